"""The paged key/value cache on the GPU (kv_append, kv_read, attn_fwd_paged) against
the 64-bit reference of tests/paged_ref.py.  Appended and read values are compared
bit for bit, attention within the bounds derived there."""
import numpy as np
import pytest
import torch

import attention_pipelining_gb300 as ap
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu

BAD_INDEX = 6


@pytest.fixture(scope="module", autouse=True)
def _built():
    ap.build()
    ap.device_status(reset=True)
    yield


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    torch.cuda.synchronize()
    assert ap.device_status(reset=True) == 0


def rng(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def tables(cap, page, seed, spare=2):
    """Random distinct pages for sequences that hold cap[b] tokens; unused entries -1."""
    blocks = [max(1, -(-c // page)) for c in cap]
    order = torch.randperm(sum(blocks) + spare, generator=rng(seed))
    bt = torch.full((len(cap), max(blocks)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        bt[b, :n] = order[at:at + n].int()
        at += n
    return bt, sum(blocks) + spare


def fill(x, fmt, kind):
    """Values [pages, H, page, D] (bf16) as a cache tensor."""
    if fmt == "bf16":
        return x.clone()
    P, H, n, D = x.shape
    b = ref.pack(ref.f64(x).reshape(-1, D), kind)
    return torch.from_numpy(b).reshape(P, H, n // 16, 9 * D)


def pools(fmt, pages, H, page, D, seed, vscale=1.0, kscale=1.0):
    g = rng(seed)
    k = fill(randn(g, pages, H, page, D, scale=kscale), fmt, "k")
    v = fill(randn(g, pages, H, page, D, scale=vscale), fmt, "v")
    return k, v


def rope(n, rot, seed=None):
    inv = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n)[:, None] * inv
    return torch.from_numpy(np.cos(a)).float(), torch.from_numpy(np.sin(a)).float()


def check_attention(q, kc, vc, bt, lens, causal, scale, got, q_lens=None, what=""):
    o, lse = (ref.f64(x) for x in got)
    kv, ks = ref.cache_values(kc, "k")
    vv, vs = ref.cache_values(vc, "v")
    page = kv.shape[2]
    ro, rl, to, tl = ref.attention(ref.f64(q), kv, vv, ks, vs, bt.cpu().numpy(), lens, page, causal,
                                   scale, q_lens)
    for b in range(q.shape[0]):
        n = q.shape[2] if q_lens is None else q_lens[b]
        a, r, t = o[b, :, :n], ro[b, :, :n], to[b, :, :n]
        assert np.isfinite(a).all(), (what, b)
        bad = np.abs(a - r) > t
        assert not bad.any(), (what, b, np.argwhere(bad)[:4], np.abs(a - r).max(), t[bad][:4])
        a, r, t = lse[b, :, :n], rl[b, :, :n], tl[b, :, :n]
        inf = np.isinf(r)
        assert np.array_equal(a[inf], r[inf]), (what, b)
        off = np.abs(a[~inf] - r[~inf])
        assert (off <= t[~inf]).all(), (what, b, off.max(), t.max())


# ---------------------------------------------------------------- append and read

APPEND = [
    # fmt, D, H_q, H_kv, S, page, starts, new_lens, rot, interleaved
    ("int4", 128, 8, 2, 1, 16, [0, 15, 16, 100], None, 128, False),
    ("int4", 128, 4, 4, 37, 32, [3, 0], None, 128, False),
    ("int4", 64, 5, 1, 20, 48, [31, 7, 0], [20, 0, 3], 64, True),
    ("int4", 64, 0, 3, 19, 16, [1], None, 32, False),
    ("int4", 128, 7, 1, 5, 64, [60, 2], None, 0, False),
    ("bf16", 128, 8, 2, 1, 16, [0, 15, 16, 100], None, 128, True),
    ("bf16", 128, 32, 8, 33, 64, [50], None, 64, False),
    ("bf16", 64, 9, 3, 21, 32, [12, 40, 0], [1, 21, 13], 64, False),
    ("bf16", 64, 2, 17, 3, 256, [254, 0], None, 16, True),
]


@pytest.mark.parametrize("case", APPEND, ids=[str(c) for c in APPEND])
def test_append_and_read(case):
    """Bit for bit: rotated queries, every byte of both pools (those not appended to
    unchanged), and what kv_read returns of them; q, k and v views of one tensor."""
    fmt, D, Hq, H, S, page, starts, new, rot, inter = case
    B = len(starts)
    counts = new or [S] * B
    cap = [s + c for s, c in zip(starts, counts)]
    bt, pages = tables(cap, page, 5)
    kc0, vc0 = pools(fmt, pages, H, page, D, 6)
    x = randn(rng(7), B, S, Hq + 2 * H, D, scale=3.0)
    x[0, 0, :, :32] = 0.0                          # a group of zeros
    x = x.transpose(1, 2)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    cos, sin = rope(max(cap) + 1, rot) if rot else (None, None)
    xd = x.cuda()
    kc, vc, btd = kc0.cuda(), vc0.cuda(), bt.cuda()
    st = torch.tensor(starts, dtype=torch.int32).cuda()
    nl = torch.tensor(new, dtype=torch.int32).cuda() if new else None
    qo = torch.full((B, Hq, S, D), 7.0, dtype=torch.bfloat16).cuda() if Hq else None
    got = ap.kv_append(xd[:, Hq:Hq + H], xd[:, Hq + H:], kc, vc, btd, st,
                       cos=cos.cuda() if rot else None, sin=sin.cuda() if rot else None,
                       q=xd[:, :Hq] if Hq else None, q_out=qo, new_lens=nl, interleaved=inter)
    torch.cuda.synchronize()
    kr, qr = ref.f64(k), ref.f64(q)
    vr = ref.f64(v)
    want_k, want_v = ref.cache_values(kc0, "k")[0], ref.cache_values(vc0, "v")[0]
    wk, wv = kc0.clone(), vc0.clone()
    for b in range(B):
        pos = starts[b] + np.arange(counts[b])
        if rot:
            c, s = cos[pos].double().numpy(), sin[pos].double().numpy()
            kb, qb = (ref.rotate(t[b, :, :counts[b]], c, s, inter) for t in (kr, qr))
        else:
            kb, qb = kr[b, :, :counts[b]], qr[b, :, :counts[b]]
        if Hq:
            assert np.array_equal(ref.f64(got[b, :, :counts[b]]), qb)
            assert (got[b, :, counts[b]:] == 7.0).all()
        for n, p in enumerate(pos):
            pg, slot = int(bt[b, p // page]), p % page
            for pool, vals, kind in ((wk, kb, "k"), (wv, vr[b], "v")):
                if fmt == "bf16":
                    pool[pg, :, slot] = torch.from_numpy(vals[:, n]).to(torch.bfloat16)
                    continue
                idx = ref.nibble_index(kind, D)[slot % 16]
                codes, sc = ref.quantise(vals[:, n])
                for h in range(H):
                    blk = pool[pg, h, slot // 16].numpy()
                    for nib, code in zip(idx, codes[h]):
                        sh = 4 * (nib % 2)
                        blk[nib // 2] = (int(blk[nib // 2]) & (0xf0 >> sh)) | (int(code) << sh)
                    at = 8 * D + slot % 16 * (D // 16)
                    blk[at:at + D // 16] = ref.to_bf16_tensor(sc[h]).view(torch.int16).numpy().view(np.uint8)
    assert torch.equal(kc.cpu(), wk) and torch.equal(vc.cpu(), wv)
    del want_k, want_v
    # read back everything, then a window that starts inside
    kv, vv = ref.cache_values(kc, "k")[0], ref.cache_values(vc, "v")[0]
    total = torch.tensor(cap, dtype=torch.int32).cuda()
    n = max(cap) + 3
    out = tuple(torch.full((B, H, n, D), 9.0, dtype=torch.bfloat16).cuda() for _ in range(2))
    ap.kv_read(kc, vc, btd, total, n, out=out)
    win = ap.kv_read(kc, vc, btd, total, S, start=st)
    torch.cuda.synchronize()
    for b in range(B):
        for vals, o, w in ((kv, out[0], win[0]), (vv, out[1], win[1])):
            want = ref.bf16(ref.gather(vals, bt[b].numpy(), cap[b], page))
            assert np.array_equal(ref.f64(o[b, :, :cap[b]]), want)
            assert (o[b, :, cap[b]:] == 9.0).all()
            assert np.array_equal(ref.f64(w[b, :, :counts[b]]), want[:, starts[b]:])
            assert (w[b, :, counts[b]:] == 0.0).all()


# ---------------------------------------------------------------- attention

ATTN = [
    # fmt, D, H_q, H_kv, S_q, page, lens, causal, q_lens
    ("int4", 128, 4, 1, 1, 16, [1], True, None),
    ("int4", 128, 8, 2, 1, 64, [500, 1, 0, 129], True, None),
    ("int4", 128, 7, 1, 1, 48, [1000], False, None),
    ("int4", 128, 16, 1, 1, 32, [333, 64], True, None),
    ("int4", 128, 32, 2, 1, 16, [700], True, None),
    ("int4", 128, 8, 2, 5, 64, [300, 4, 3, 0], True, None),
    ("int4", 128, 4, 4, 3, 16, [129, 257], False, [2, 3]),
    ("int4", 128, 6, 2, 40, 32, [40, 100], True, [40, 17]),
    ("int4", 128, 20, 1, 2, 16, [1300, 200], True, None),
    ("int4", 128, 32, 1, 2, 48, [95, 0, 600], False, None),
    ("int4", 64, 4, 1, 1, 16, [2500, 15, 16, 17], True, None),
    ("int4", 64, 12, 1, 1, 256, [1025], True, None),
    ("int4", 64, 4, 2, 9, 16, [77, 8], True, [9, 0]),
    ("int4", 64, 3, 3, 30, 16, [64], True, None),
    ("bf16", 128, 8, 2, 1, 64, [500, 1, 0, 129], True, None),
    ("bf16", 128, 16, 1, 1, 48, [333, 48], True, None),
    ("bf16", 128, 24, 1, 1, 16, [700], True, None),
    ("bf16", 128, 8, 2, 5, 16, [300, 4, 3, 0], True, None),
    ("bf16", 128, 6, 2, 40, 32, [40, 100], True, [40, 17]),
    ("bf16", 128, 16, 1, 4, 64, [1300, 200], True, None),
    ("bf16", 64, 48, 1, 1, 16, [95, 0, 600], False, None),
    ("bf16", 64, 4, 1, 1, 16, [2500, 15, 16, 17], False, None),
    ("bf16", 64, 4, 2, 9, 16, [77, 8], True, [9, 0]),
    ("bf16", 64, 3, 3, 30, 32, [64, 65], True, None),
]


@pytest.mark.parametrize("case", ATTN, ids=[str(c) for c in ATTN])
def test_attention(case):
    fmt, D, Hq, H, Sq, page, lens, causal, q_lens = case
    B = len(lens)
    bt, pages = tables([max(n, 1) for n in lens], page, 11)
    kc, vc = pools(fmt, pages, H, page, D, 12)
    q = randn(rng(13), B, Hq, Sq, D, scale=1.5)
    scale = D ** -0.5
    out = (torch.full((B, Hq, Sq, D), 5.0, dtype=torch.bfloat16).cuda(),
           torch.full((B, Hq, Sq), 5.0).cuda())
    ql = torch.tensor(q_lens, dtype=torch.int32).cuda() if q_lens else None
    kd, vd, bd = kc.cuda(), vc.cuda(), bt.cuda()
    ld = torch.tensor(lens, dtype=torch.int32).cuda()
    ap.attn_fwd_paged(q.cuda(), kd, vd, bd, ld, causal, scale, q_lens=ql, out=out)
    torch.cuda.synchronize()
    check_attention(q, kc, vc, bt, lens, causal, scale, out, q_lens, str(case))
    for b in range(B):
        n = Sq if q_lens is None else q_lens[b]
        assert (out[0][b, :, n:] == 5.0).all() and (out[1][b, :, n:] == 5.0).all()
    # block tables that span more keys than an item is kept whole for
    wide = torch.cat([bt, torch.full((B, 1024 // page + 1), -1, dtype=torch.int32)], 1)
    split = tuple(torch.full_like(t, 5.0) for t in out)
    ap.attn_fwd_paged(q.cuda(), kd, vd, wide.cuda(), ld, causal, scale, q_lens=ql, out=split)
    torch.cuda.synchronize()
    check_attention(q, kc, vc, bt, lens, causal, scale, split, q_lens, str(case) + " split")
    for b in range(B):
        n = Sq if q_lens is None else q_lens[b]
        assert (split[0][b, :, n:] == 5.0).all() and (split[1][b, :, n:] == 5.0).all()
    # the same bits again, from a strided q
    qs = q.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    o2, l2 = ap.attn_fwd_paged(qs, kd, vd, bd, ld, causal, scale, q_lens=ql)
    for b in range(B):
        n = Sq if q_lens is None else q_lens[b]
        assert torch.equal(o2[b, :, :n], out[0][b, :, :n]) and torch.equal(l2[b, :, :n], out[1][b, :, :n])


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_long_and_ragged_batch(fmt):
    """Sequences that many thread blocks share next to short ones, and more sequences
    than a plan thread's one."""
    lens = [20000, 3, 0, 511] + [(37 * i) % 200 for i in range(140)]
    D, Hq, H, page = 64, 4, 2, 32
    bt, pages = tables([max(n, 1) for n in lens], page, 21)
    kc, vc = pools(fmt, pages, H, page, D, 22, vscale=0.02)
    q = randn(rng(23), len(lens), Hq, 1, D)
    got = ap.attn_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), bt.cuda(),
                            torch.tensor(lens, dtype=torch.int32).cuda(), True, 0.2)
    check_attention(q, kc, vc, bt, lens, True, 0.2, got, what=fmt)
