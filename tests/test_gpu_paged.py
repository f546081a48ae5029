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


# ---------------------------------------------------------------- what must not matter


def device_ints(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def spoil(pool, bt, lens, page, inside=None):
    """A copy whose slots behind the sequences' ends, and pages of no sequence, hold NaN and
    infinities (bf16) or bytes of ones (4 bits: codes 15 and NaN scales)."""
    bad = torch.full_like(pool, 255) if pool.dtype == torch.uint8 else \
        torch.where(torch.rand(pool.shape, generator=rng(99)) < 0.5, float("nan"), float("inf")).to(pool.dtype)
    D = pool.shape[3] // 9 if pool.dtype == torch.uint8 else pool.shape[3]
    for b, L in enumerate(lens):
        for x in range(L):
            pg, slot = int(bt[b, x // page]), x % page
            if pool.dtype != torch.uint8:
                bad[pg, :, slot] = pool[pg, :, slot]
                continue
            for kind in (inside,):
                byte = np.unique(ref.nibble_index(kind, D)[slot % 16] // 2)
                byte = np.concatenate([byte, 8 * D + slot % 16 * (D // 16) + np.arange(D // 16)])
                bad[pg, :, slot // 16, byte] = pool[pg, :, slot // 16, byte]
    return bad


@pytest.mark.parametrize("Sq", [1, 5])
@pytest.mark.parametrize("fmt,D", [("int4", 128), ("int4", 64), ("bf16", 128), ("bf16", 64)])
def test_what_lies_behind_the_end_does_not_matter(fmt, D, Sq):
    lens, page = [77, 16, 5, 33], 32
    bt, pages = tables(lens, page, 31)
    kc, vc = pools(fmt, pages, 2, page, D, 32)
    q = randn(rng(33), 4, 6, Sq, D)
    n = device_ints(*lens)
    want = ap.attn_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), bt.cuda(), n, True, 0.1)
    kb, vb = spoil(kc, bt, lens, page, "k"), spoil(vc, bt, lens, page, "v")
    for wide in (bt, torch.cat([bt, torch.full((4, 64), 2 ** 30, dtype=torch.int32)], 1)):
        got = ap.attn_fwd_paged(q.cuda(), kb.cuda(), vb.cuda(), wide.cuda(), n, True, 0.1)
        if wide is bt:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        check_attention(q, kc, vc, bt, lens, True, 0.1, got)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("fmt,D,Hq", [("int4", 64, 4), ("bf16", 128, 2), ("bf16", 64, 12)])
def test_a_value_that_a_row_does_not_see_does_not_matter(fmt, D, Hq, bad):
    """The last token's key and value are not finite: of four causal queries only the last one
    sees them."""
    L, page = 45, 16
    bt, pages = tables([L], page, 41)
    g = rng(42)
    k, v = randn(g, pages, 1, page, D), randn(g, pages, 1, page, D)
    kc, vc = fill(k, fmt, "k"), fill(v, fmt, "v")
    pg, slot = int(bt[0, (L - 1) // page]), (L - 1) % page
    k[pg, 0, slot], v[pg, 0, slot, ::3] = bad, bad
    kn, vn = fill(k, fmt, "k"), fill(v, fmt, "v")
    q = randn(g, 1, Hq, 4, D)
    o, lse = ap.attn_fwd_paged(q.cuda(), kn.cuda(), vn.cuda(), bt.cuda(), device_ints(L), True, 0.1)
    head = (o[:, :, :3].contiguous(), lse[:, :, :3].contiguous())
    check_attention(q[:, :, :3], kc, vc, bt, [L - 1], True, 0.1, head)
    assert not torch.isfinite(o[0, :, 3]).all()


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_a_sequence_s_nan_stays_its_own(fmt):
    """A NaN key in one sequence: its rows are NaN, the others' as without."""
    lens, page, D = [100, 300, 40], 16, 64
    bt, pages = tables(lens, page, 43)
    g = rng(44)
    k, v = randn(g, pages, 2, page, D), randn(g, pages, 2, page, D)
    q = randn(g, 3, 4, 1, D)
    bad = k.clone()
    bad[int(bt[1, 7]), 1, 3, 9] = float("nan")
    vc = fill(v, fmt, "v")
    a, _ = ap.attn_fwd_paged(q.cuda(), fill(k, fmt, "k").cuda(), vc.cuda(), bt.cuda(),
                             device_ints(*lens), True, 0.1)
    b, _ = ap.attn_fwd_paged(q.cuda(), fill(bad, fmt, "k").cuda(), vc.cuda(), bt.cuda(),
                             device_ints(*lens), True, 0.1)
    assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1, :2], b[1, :2])
    assert torch.isnan(b[1, 2:]).all()


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_page_numbers_out_of_range(fmt):
    """Such pages are never followed: their keys are masked, their tokens neither written nor
    read, and the status word says so."""
    L, page, D, H = 200, 16, 64, 2
    bt, pages = tables([L, L], page, 51)
    kc, vc = pools(fmt, pages, H, page, D, 52)
    bad = bt.clone()
    bad[0, 2], bad[0, 7], bad[1, 12] = -1, pages, 2 ** 31 - 1
    q = randn(rng(53), 2, 4, 1, D)
    got = ap.attn_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), bad.cuda(), device_ints(L, L), False, 0.1)
    torch.cuda.synchronize()
    assert ap.device_status(reset=True) == BAD_INDEX
    for b, gone in ((0, (2, 7)), (1, (12,))):
        keep = torch.tensor([[int(p) for i, p in enumerate(bt[b]) if i not in gone]], dtype=torch.int32)
        n = L - sum(min(page, L - i * page) for i in gone)
        check_attention(q[b:b + 1], kc, vc, keep, [n], False, 0.1, [t[b:b + 1] for t in got])
    # read: the rows of missing pages stay as they were
    out = tuple(torch.full((2, H, L, D), 3.0, dtype=torch.bfloat16).cuda() for _ in range(2))
    ap.kv_read(kc.cuda(), vc.cuda(), bad.cuda(), device_ints(L, L), L, out=out)
    torch.cuda.synchronize()
    assert ap.device_status(reset=True) == BAD_INDEX
    full = ap.kv_read(kc.cuda(), vc.cuda(), bt.cuda(), device_ints(L, L), L)
    for got_t, want in zip(out, full):
        want[0, :, 32:48], want[0, :, 112:128], want[1, :, 192:] = 3.0, 3.0, 3.0
        assert torch.equal(got_t, want)
    # append: tokens 190 .. 195 of sequence 1 reach into its missing page
    k = randn(rng(54), 2, H, 6, D).cuda()
    qo = torch.full((2, 3, 6, D), 4.0, dtype=torch.bfloat16).cuda()
    k1, v1 = kc.cuda(), vc.cuda()
    ap.kv_append(k, k, k1, v1, bad.cuda(), device_ints(50, 190), q=randn(rng(55), 2, 3, 6, D).cuda(), q_out=qo)
    torch.cuda.synchronize()
    assert ap.device_status(reset=True) == BAD_INDEX
    k2, v2 = kc.cuda(), vc.cuda()
    ap.kv_append(k, k, k2, v2, bt.cuda(), device_ints(50, 190), new_lens=device_ints(6, 2))
    torch.cuda.synchronize()
    assert torch.equal(k1, k2) and torch.equal(v1, v2)
    assert (qo[1, :, 2:] == 4.0).all() and not (qo[:, :, :2] == 4.0).all()


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_lengths_out_of_range_are_cut(fmt):
    page, D = 16, 64
    bt, pages = tables([64, 64, 64], page, 56)
    kc, vc = (t.cuda() for t in pools(fmt, pages, 1, page, D, 57))
    q = randn(rng(58), 3, 2, 2, D).cuda()
    want = ap.attn_fwd_paged(q, kc, vc, bt.cuda(), device_ints(0, 64, 40), True, 0.1,
                             q_lens=device_ints(2, 2, 0))
    torch.cuda.synchronize()
    assert ap.device_status(reset=True) == 0
    for lens, ql in (((-7, 64, 40), (2, 2, 0)), ((0, 65, 40), (2, 2, 0)), ((0, 64, 40), (2, 3, -1))):
        got = ap.attn_fwd_paged(q, kc, vc, bt.cuda(), device_ints(*lens), True, 0.1,
                                q_lens=device_ints(*ql))
        torch.cuda.synchronize()
        assert ap.device_status(reset=True) == BAD_INDEX
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # positions before the cache or behind its end, or without a rotation, are skipped
    cos, sin = (t.cuda() for t in rope(40, D))
    k = randn(rng(59), 3, 1, 4, D).cuda()
    before = kc.clone()
    ap.kv_append(k, k, kc, vc, bt.cuda(), device_ints(-4, 64, 40), cos=cos, sin=sin)
    torch.cuda.synchronize()
    assert ap.device_status(reset=True) == BAD_INDEX
    assert torch.equal(kc, before)


def test_scores_of_any_size():
    """Large, tiny, negative and zero softmax scales; keys and values whose scales differ by
    many powers of two from token to token; a row of zeros and one of tiny queries."""
    L, page, D = 300, 48, 128
    bt, pages = tables([L], page, 61)
    g = rng(62)
    span = torch.exp2(torch.randint(-12, 9, (pages, 1, page, 1), generator=g).float())
    k = (torch.randn((pages, 1, page, D), generator=g) * span).to(torch.bfloat16)
    v = (torch.randn((pages, 1, page, D), generator=g) * span.flip(2)).to(torch.bfloat16)
    q = randn(g, 1, 6, 1, D)
    q[0, 1], q[0, 2], q[0, 3] = 0.0, q[0, 2] * 2.0 ** -100, q[0, 3] * 2.0 ** 20
    for fmt in ("int4", "bf16"):
        kc, vc = fill(k, fmt, "k"), fill(v, fmt, "v")
        for scale in (0.001, -0.002, 0.0, 1e-30):
            got = ap.attn_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), bt.cuda(), device_ints(L), False, scale)
            check_attention(q, kc, vc, bt, [L], False, scale, got, what=(fmt, scale))
        # the largest scale that is finite: nothing breaks down
        o, _ = ap.attn_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), bt.cuda(), device_ints(L), False, 3.4e38)
        assert torch.isfinite(o[0, 1]).all()


# ---------------------------------------------------------------- rounding of the rotation


def test_rotation_rounds_the_exact_value():
    """Two million rotated elements, bit for bit, and sums next to a tie of the rounding that
    only the products' lowest bits decide."""
    S, H, D = 2048, 8, 128
    x = randn(rng(71), 1, H, S, D, scale=2.0)
    cos, sin = rope(S, D)
    kc, vc = ap.kv_cache_empty(S // 64, H, 64, D)
    bt = torch.arange(S // 64, dtype=torch.int32)[None].cuda()
    xd = x.cuda()
    ap.kv_append(xd, xd, kc, vc, bt, device_ints(0), cos=cos.cuda(), sin=sin.cuda())
    got = ap.kv_read(kc, vc, bt, device_ints(S), S)[0]
    want = ref.rotate(ref.f64(x), cos.double().numpy(), sin.double().numpy(), False)
    assert np.array_equal(ref.f64(got), want)
    # x cos is a tie of the rounding to 8 bits; y sin moves it by less than fp32 holds
    t = np.array([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 129 * 2.0 ** -7 + 2.0 ** -8])
    d = np.array([0.0, 2.0 ** -30, -2.0 ** -30, 2.0 ** -40, -2.0 ** -40])
    cos2 = np.repeat(t, len(d))[:, None] * np.ones((1, 8))
    sin2 = np.tile(d, len(t))[:, None] * np.ones((1, 8))
    n = len(cos2)
    one = torch.ones((1, 1, n, 64), dtype=torch.bfloat16)
    kc, vc = ap.kv_cache_empty(1, 1, 16, 64)
    for sign in (1.0, -1.0):
        y = (one * sign).cuda()
        ap.kv_append(y, y, kc, vc, bt[:, :1], device_ints(0), cos=torch.from_numpy(cos2).float().cuda(),
                     sin=torch.from_numpy(sin2).float().cuda(), interleaved=True)
        got = ref.f64(kc[0, 0, :n, :16])
        a = sign * np.repeat(cos2, 2, 1)
        b = sign * np.stack([-sin2, sin2], -1).reshape(n, 16)
        want = ref.bf16(a)
        tie = np.abs(a) * 256 % 2 == 1
        up = np.sign(a) * (2.0 ** -8)
        want = np.where(b == 0, want, np.where(np.sign(b) == np.sign(a), a + up, a - up))
        assert tie.all() and np.array_equal(got, want)


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_append_of_values_that_are_not_finite(fmt):
    """A 4-bit group with an infinity or a NaN reads as NaN, the others as ever; bf16 keeps them;
    a rotated infinity is the formula's."""
    D, S = 64, 3
    x = randn(rng(73), 1, 1, S, D)
    x[0, 0, 0, 5], x[0, 0, 1, 40] = float("inf"), float("nan")
    kc, vc = ap.kv_cache_empty(1, 1, 16, D, fmt)
    bt = torch.zeros((1, 1), dtype=torch.int32).cuda()
    cos, sin = torch.full((16, 8), 0.5).cuda(), torch.full((16, 8), 0.25).cuda()
    q = ap.kv_append(x.cuda(), x.cuda(), kc, vc, bt, device_ints(0), cos=cos, sin=sin, q=x.cuda())
    k, v = ap.kv_read(kc, vc, bt, device_ints(S), S)
    q, k, v = q.cpu(), k.cpu(), v.cpu()
    assert q[0, 0, 0, 5] == float("inf") and q[0, 0, 0, 13] == float("inf")   # x .5, x .25 of the pair
    assert torch.isnan(q[0, 0, 1, 40]) and torch.isfinite(q[0, 0, 2]).all()
    if fmt == "bf16":
        assert torch.equal(v.isnan(), x.isnan()) and torch.equal(v.isinf(), x.isinf())
        return
    assert v[0, 0, 0, :32].isnan().all() and v[0, 0, 1, 32:].isnan().all()
    assert v[0, 0, 0, 32:].isfinite().all() and v[0, 0, 1, :32].isfinite().all()
    assert v[0, 0, 2].isfinite().all() and k[0, 0, 2].isfinite().all()


def test_quantisation_of_every_ratio():
    """Codes of all pairs (element, largest of the group) of 8-bit mantissas on both sides of a
    power of two, ties among them; groups whose scale is subnormal or 0; bit for bit."""
    D = 64
    m = np.arange(128, 256) / 128.0
    x = np.concatenate([m, m / 2, m / 4, m / 8])
    vals = np.zeros((len(m), 17, 32))   # each group: its largest element and 31 others
    for i, top in enumerate(m):
        others = np.zeros(17 * 31)
        others[:len(x)] = np.minimum(x, top)
        vals[i, :, 0] = top
        vals[i, :, 1:] = others.reshape(17, 31) * np.where(np.arange(31) % 2, 1, -1)
    vals = vals.reshape(-1, D)
    vals = np.concatenate([vals, vals[::7] * 2.0 ** -98, vals[::7] * 2.0 ** -120,
                           vals[::7] * 2.0 ** -126, vals[::7] * 2.0 ** -131])
    S = len(vals)
    v = torch.from_numpy(vals).to(torch.bfloat16)[None, None]
    kc, vc = ap.kv_cache_empty(-(-S // 64), 1, 64, D, "int4")
    vc.zero_()
    bt = torch.arange(kc.shape[0], dtype=torch.int32)[None].cuda()
    ap.kv_append(v.cuda(), v.cuda(), kc, vc, bt, device_ints(0))
    torch.cuda.synchronize()
    f = ref.f64(v)[0, 0]
    # float64 division and torch's rounding of the scale to bf16 (subnormals too)
    g = f.reshape(-1, 2, 32)
    s = torch.from_numpy(np.abs(g).max(-1) / 7).to(torch.bfloat16).double().numpy()
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.where(s[..., None] > 0, np.clip(np.round(g / s[..., None]), -7, 7), 0) + 8
    code = code.astype(np.uint8).reshape(S, D)
    got = vc.cpu().numpy().reshape(-1, 9 * D)
    idx = ref.nibble_index("v", D)
    for t in range(S):
        blk = got[t // 16]
        nib = (blk[idx[t % 16] // 2] >> (4 * (idx[t % 16] % 2))) & 15
        assert np.array_equal(nib, code[t]), t


MERGE = [
    # fmt, D, H_q, H_kv, S_q, lens, causal, q_lens: few items of many parts, down to one part
    ("int4", 128, 4, 1, 1, [9000], True, None),
    ("int4", 64, 8, 2, 5, [6000, 0, 130], True, [5, 5, 2]),
    ("int4", 128, 2, 2, 1, [1, 7001], False, None),
    ("bf16", 128, 6, 1, 9, [8000, 40], True, [9, 0]),
    ("bf16", 64, 1, 1, 100, [5000], True, None),
    ("bf16", 128, 3, 3, 1, [4097], False, None),
    # many items, two or three parts each
    ("int4", 128, 16, 16, 2, [1200, 900, 1, 1090, 0], True, [2, 1, 1, 2, 2]),
    ("bf16", 64, 40, 20, 1, [1100, 1300, 1290, 7], False, None),
]


@pytest.mark.parametrize("case", MERGE, ids=[str(c) for c in MERGE])
def test_parts_of_items(case):
    """Items on one to hundreds of thread blocks; a workspace full of NaN and of every bit set;
    rows of padding stay as they were."""
    fmt, D, Hq, H, Sq, lens, causal, q_lens = case
    B, page = len(lens), 64
    bt, pages = tables([max(n, 1) for n in lens], page, 91)
    kc, vc = pools(fmt, pages, H, page, D, 92)
    q = randn(rng(93), B, Hq, Sq, D)
    n = ap.paged_workspace_bytes(B, Hq, H, Sq, D, bt.shape[1] * page)
    results = []
    for fill_with in (0xff, 0x7f):
        ws = torch.full((n,), fill_with, dtype=torch.uint8).cuda()
        out = (torch.full((B, Hq, Sq, D), 3.0, dtype=torch.bfloat16).cuda(),
               torch.full((B, Hq, Sq), 3.0).cuda())
        got = ap.attn_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), bt.cuda(), device_ints(*lens), causal,
                                0.3, q_lens=device_ints(*q_lens) if q_lens else None, workspace=ws,
                                out=out)
        torch.cuda.synchronize()
        results.append([x.cpu() for x in got])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    check_attention(q, kc, vc, bt, lens, causal, 0.3, results[0], q_lens, what=str(case))
    for b in range(B if q_lens else 0):
        assert (results[0][0][b, :, q_lens[b]:] == 3).all() and (results[0][1][b, :, q_lens[b]:] == 3).all()


# ---------------------------------------------------------------- together, as used


@pytest.mark.parametrize("fmt,D,Hq,H", [("int4", 128, 8, 2), ("bf16", 64, 6, 3)])
def test_prompts_then_decoding(fmt, D, Hq, H):
    """Two prompts of different lengths go into the cache and get their attention from what the
    cache holds; then both sequences grow token by token, a captured graph of one step replayed
    while the lengths advance on the device.  Every step against the 64-bit attention over
    everything appended so far, and bit for bit against uncaptured calls."""
    page, steps, prompt = 16, 9, [37, 12]
    cap = [n + steps for n in prompt]
    bt, pages = tables(cap, page, 81)
    bt = torch.cat([bt, torch.full((2, 70), -1, dtype=torch.int32)], 1)     # room that splits items
    btd = bt.cuda()
    g = rng(82)
    cos, sin = (t.cuda() for t in rope(128, D))
    scale = D ** -0.5
    kc, vc = ap.kv_cache_empty(pages, H, page, D, fmt)
    kc.fill_(255 if fmt == "int4" else float("nan"))
    vc.fill_(255 if fmt == "int4" else float("nan"))
    S = max(prompt)
    x = randn(g, 2, S, Hq + 2 * H, D).transpose(1, 2).cuda()
    lens = device_ints(*prompt)
    q = ap.kv_append(x[:, Hq:Hq + H], x[:, Hq + H:], kc, vc, btd, device_ints(0, 0), cos=cos, sin=sin,
                     q=x[:, :Hq], new_lens=lens)
    o, lse = ap.attn_fwd_paged(q, kc, vc, btd, lens, True, scale, q_lens=lens)
    check_attention(q.cpu(), kc, vc, bt, prompt, True, scale, (o, lse), prompt, "prompt")
    # the same through the framework's prompt attention on what kv_read returns
    k, v = ap.kv_read(kc, vc, btd, lens, S)
    for b, n in enumerate(prompt):
        ob, lb = ap.attn_fwd(q[b:b + 1, :, :n].contiguous(), k[b:b + 1, :, :n].contiguous(),
                             v[b:b + 1, :, :n].contiguous(), True, scale)
        assert (ob.float() - o[b:b + 1, :, :n].float()).abs().max() <= 0.03
        assert (lb - lse[b:b + 1, :, :n]).abs().max() <= 0.02
    # decoding
    new = torch.empty((2, 1, Hq + 2 * H, D), dtype=torch.bfloat16).cuda().transpose(1, 2)
    start, total = lens.clone(), lens + 1
    ws = torch.empty(ap.paged_workspace_bytes(2, Hq, H, 1, D, bt.shape[1] * page), dtype=torch.uint8).cuda()
    q1 = torch.empty((2, Hq, 1, D), dtype=torch.bfloat16).cuda()
    out = (torch.empty_like(q1), torch.empty((2, Hq, 1)).cuda())

    def step():
        ap.kv_append(new[:, Hq:Hq + H], new[:, Hq + H:], kc, vc, btd, start, cos=cos, sin=sin,
                     q=new[:, :Hq], q_out=q1)
        ap.attn_fwd_paged(q1, kc, vc, btd, total, True, scale, workspace=ws, out=out)
        start.add_(1)
        total.add_(1)

    tokens = [randn(g, 2, Hq + 2 * H, 1, D) for _ in range(steps)]
    new.copy_(tokens[0].cuda())
    saved = kc.clone(), vc.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    assert torch.equal(start, lens)                      # captured, not run
    got = []
    for i in range(steps):
        new.copy_(tokens[i].cuda())
        graph.replay()
        torch.cuda.synchronize()
        got.append((q1.clone(), out[0].clone(), out[1].clone()))
        now = [n + i + 1 for n in prompt]
        check_attention(q1.cpu(), kc, vc, bt, now, True, scale, out, what=i)
    assert start.tolist() == [n + steps for n in prompt]
    final = kc.clone(), vc.clone()
    kc.copy_(saved[0]), vc.copy_(saved[1])
    start.copy_(lens), total.copy_(lens + 1)
    for i in range(steps):
        new.copy_(tokens[i].cuda())
        step()
        assert torch.equal(q1, got[i][0]) and torch.equal(out[0], got[i][1]) and torch.equal(out[1], got[i][2])
    torch.cuda.synchronize()
    assert torch.equal(kc.view(torch.uint8), final[0].view(torch.uint8))
    assert torch.equal(vc.view(torch.uint8), final[1].view(torch.uint8))


def test_cross_attention_to_encoder_states():
    """Two decoders' queries over encoder states of other lengths, kept in the cache unrotated,
    and without a mask."""
    D, H, enc, page = 64, 4, [93, 20], 32
    bt, pages = tables(enc, page, 83)
    kc, vc = ap.kv_cache_empty(pages, H, page, D)
    kc.zero_(), vc.zero_()
    k, v = (randn(rng(84 + i), 2, H, max(enc), D).cuda() for i in range(2))
    n = device_ints(*enc)
    assert ap.kv_append(k, v, kc, vc, bt.cuda(), device_ints(0, 0), new_lens=n) is None
    q = randn(rng(86), 2, H, 7, D)
    got = ap.attn_fwd_paged(q.cuda(), kc, vc, bt.cuda(), n, False, 0.125)
    check_attention(q, kc, vc, bt, enc, False, 0.125, got)
    for b, m in enumerate(enc):
        assert torch.equal(ap.kv_read(kc, vc, bt.cuda(), n, m)[1][b], v[b, :, :m])


def test_streams_shared_pages_and_two_calls_at_once():
    """Sequences that share pages; calls on two streams at once, each with its own workspace,
    and one without; the bits are those of a single call."""
    D, H, page, L = 128, 2, 64, 3000
    bt, pages = tables([L], page, 87)
    bt = bt.repeat(6, 1)                       # six sequences, one set of pages
    kc, vc = (t.cuda() for t in pools("int4", pages, H, page, D, 88))
    lens = [L, 1, 700, 0, 2999, 64]
    q = randn(rng(89), 6, 8, 1, D)
    n = device_ints(*lens)
    qd, btd = q.cuda(), bt.cuda()
    want = ap.attn_fwd_paged(qd, kc, vc, btd, n, True, 0.1)
    check_attention(q, kc, vc, bt, lens, True, 0.1, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    ws = [torch.full((ap.paged_workspace_bytes(6, 8, H, 1, D, bt.shape[1] * page),), 255,
                     dtype=torch.uint8).cuda() for _ in range(2)] + [None]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got += [ap.attn_fwd_paged(qd, kc, vc, btd, n, True, 0.1, workspace=w, stream=s)
                for s, w in zip(streams, ws)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in got)


def test_graphs_with_their_own_workspaces():
    """Two captured graphs, replayed in turn and on two streams at once."""
    D, H, page, L = 64, 1, 16, 4000
    bt, pages = tables([L], page, 91)
    kc, vc = (t.cuda() for t in pools("bf16", pages, H, page, D, 92))
    btd, n = bt.cuda(), device_ints(L)
    qs = [randn(rng(93 + i), 1, 4, 1, D).cuda() for i in range(2)]
    want = [ap.attn_fwd_paged(q, kc, vc, btd, n, True, 0.1) for q in qs]
    graphs, outs, keep = [], [], []
    for q in qs:
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        out = (torch.empty_like(q), torch.empty((1, 4, 1)).cuda())
        ws = torch.empty(ap.paged_workspace_bytes(1, 4, H, 1, D, bt.shape[1] * page), dtype=torch.uint8).cuda()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            ap.attn_fwd_paged(q, kc, vc, btd, n, True, 0.1, workspace=ws, out=out)
        graphs.append(g), outs.append(out), keep.append((s, ws))
    for _ in range(3):
        for (s, _), g, out in zip(keep, graphs, outs):
            with torch.cuda.stream(s):
                out[0].zero_()
                g.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])


def test_workspace_that_the_call_allocates():
    """It belongs to the call's stream, and in a captured call to the graph: memory that others get
    meanwhile is other memory."""
    D, H, page, L = 128, 2, 32, 30000
    bt, pages = tables([L], page, 96)
    kc, vc = (t.cuda() for t in pools("int4", pages, H, page, D, 97))
    btd, n = bt.cuda(), device_ints(L)
    q = randn(rng(98), 1, 8, 1, D).cuda()
    size = ap.paged_workspace_bytes(1, 8, H, 1, D, bt.shape[1] * page)
    want = ap.attn_fwd_paged(q, kc, vc, btd, n, True, 0.1)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    s = torch.cuda.Stream()
    outs = [(torch.zeros_like(q), torch.zeros((1, 8, 1)).cuda()) for _ in range(8)]
    torch.cuda.synchronize()
    for out in outs:
        ap.attn_fwd_paged(q, kc, vc, btd, n, True, 0.1, out=out, stream=s)
        for _ in range(4):
            torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for out in outs[:2]:
            ap.attn_fwd_paged(q, kc, vc, btd, n, True, 0.1, out=out)
    for _ in range(5):
        outs[0][0].zero_(), outs[1][0].zero_()
        g.replay()
        held = [torch.full((size,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        for out in outs[:2]:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert all((x == 0xff).all() for x in held)
    del held, out, outs
    # (a workspace still held would be `size` more; the graph itself holds two small blocks)
    after = torch.cuda.memory_allocated()
    assert after < before + size
    with pytest.raises(ap.AttnError):   # refused after it was allocated: freed all the same
        ap.attn_fwd_paged(q, kc, vc, btd, n, True, float("inf"))
    assert torch.cuda.memory_allocated() == after


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_pools_larger_than_32_bit_offsets(fmt):
    """The sequence's pages are the last of a pool of more than 2^32 bytes."""
    H, page, D, L = 8, 64, 128, 300
    per = H * page * (D * 2 if fmt == "bf16" else 72)
    pages = (1 << 32) // per + 40
    kc, vc = ap.kv_cache_empty(pages, H, page, D, fmt)
    bt = torch.arange(pages - 1, pages - 6, -1, dtype=torch.int32)[None].cuda()
    k, v = (randn(rng(95 + i), 1, H, L, D).cuda() for i in range(2))
    ap.kv_append(k, v, kc, vc, bt, device_ints(0))
    small = tuple(t[pages - 5:].clone() for t in (kc, vc))
    q = randn(rng(97), 1, 8, 1, D)
    near = torch.tensor([[4, 3, 2, 1, 0]], dtype=torch.int32)
    got = ap.attn_fwd_paged(q.cuda(), kc, vc, bt, device_ints(L), True, 0.09)
    check_attention(q, *small, near, [L], True, 0.09, got)
    if fmt == "bf16":
        back = ap.kv_read(kc, vc, bt, device_ints(L), L)
        assert torch.equal(back[0], k) and torch.equal(back[1], v)


def test_one_very_long_sequence():
    """131072 4-bit keys of one head over many thread blocks."""
    L, page, D = 131072, 256, 64
    bt, pages = tables([L], page, 98, spare=0)
    g = torch.Generator().manual_seed(99)
    kc = torch.randint(0, 256, (pages, 1, page // 16, 9 * D), generator=g, dtype=torch.uint8)
    vc = torch.randint(0, 256, (pages, 1, page // 16, 9 * D), generator=g, dtype=torch.uint8)
    for t in (kc, vc):   # scales of about 1 / 8, positive
        s = (torch.rand(t.shape[:3] + (D // 2,), generator=g) * 0.1 + 0.1).to(torch.bfloat16)
        t[..., 8 * D:] = s.view(torch.uint8)
    q = randn(rng(100), 1, 5, 1, D)
    got = ap.attn_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), bt.cuda(), device_ints(L), True, 0.125)
    check_attention(q, kc, vc, bt, [L], True, 0.125, got)


def test_refusals_on_the_device():
    D = 64
    kc, vc = ap.kv_cache_empty(4, 2, 16, D, "int4")
    kb, vb = ap.kv_cache_empty(4, 2, 16, D)
    bt = torch.zeros((2, 80), dtype=torch.int32).cuda()
    n = device_ints(1, 1)
    q = torch.zeros((2, 4, 1, D), dtype=torch.bfloat16).cuda()
    k = torch.zeros((2, 2, 1, D), dtype=torch.bfloat16).cuda()
    f = ap.attn_fwd_paged
    with pytest.raises(TypeError):
        f(q.half(), kb, vb, bt, n, True, 0.1)
    with pytest.raises(ValueError):
        f(q, kb, vc, bt, n, True, 0.1)
    with pytest.raises(TypeError):
        f(q, kb, vb, bt.long(), n, True, 0.1)
    with pytest.raises(TypeError):
        f(q, kb, vb, bt, n.long(), True, 0.1)
    with pytest.raises(TypeError):
        f(q, kb, vb, bt, n[:1], True, 0.1)
    with pytest.raises(ValueError):
        f(q[:1], kb, vb, bt, n, True, 0.1)
    with pytest.raises(ap.AttnError):
        f(q[:, :3], kb, vb, bt, n, True, 0.1)                    # three heads over two
    with pytest.raises(ap.AttnError):
        f(q, kb, vb, bt, n, True, float("nan"))
    with pytest.raises(ap.AttnError):
        f(q, kb, vb, bt, n, True, 0.1, workspace=torch.empty(64, dtype=torch.uint8).cuda())
    with pytest.raises(TypeError):
        f(q, kb, vb, bt, n, True, 0.1, out=(q, torch.empty(2, 4).cuda()))
    odd = torch.zeros((2, 4, 1, D + 4), dtype=torch.bfloat16).cuda()[..., 4:]
    with pytest.raises(ap.AttnError):
        f(odd, kb, vb, bt, n, True, 0.1)                          # 8 bytes off, strides of 68
    with pytest.raises(ValueError):
        ap.kv_append(k.expand(2, 2, 1, D).transpose(2, 3), k, kc, vc, bt, n)
    with pytest.raises(ValueError):
        ap.kv_append(k, k, kc, vc, bt, n, cos=torch.zeros(9, 0).cuda(), sin=torch.zeros(9, 0).cuda())
    with pytest.raises(ap.AttnError):
        ap.kv_append(k, k, kc, vc, bt, n, cos=torch.zeros(9, 4).cuda(), sin=torch.zeros(9, 4).cuda())
    with pytest.raises(TypeError):
        ap.kv_append(k, k, kc, vc, bt, n, cos=torch.zeros(9, 8).cuda())
    with pytest.raises(ValueError):
        ap.kv_append(k, k, kc, vc, bt, n, q_out=q)
    with pytest.raises(TypeError):
        ap.kv_read(kc, vc, bt, n, 4, out=(k, k))
    with pytest.raises(ap.AttnError):
        ap.kv_read(kc, vc, bt, n, 0)


# ---------------------------------------------------------------- failure detection


@pytest.mark.parametrize("fmt,D,Hq", [("int4", 128, 4), ("int4", 64, 20), ("bf16", 128, 4), ("bf16", 64, 64)])
def test_a_wait_that_runs_out(fmt, D, Hq):
    """One stage of keys and values is never requested: every warp stops, the status word reads
    ATTN_ERR_TIMEOUT, and the same call right after is right."""
    L, page = 5000, 16
    bt, pages = tables([L], page, 101)
    kc, vc = pools(fmt, pages, 1, page, D, 102)
    q = randn(rng(103), 1, Hq, 1, D)
    args = (q.cuda(), kc.cuda(), vc.cuda(), bt.cuda(), device_ints(L), True, 0.1)
    ap.paged.fwd_paged_timeout_test(*args, drop_stage=0, wait_budget_ns=20_000_000)
    torch.cuda.synchronize()
    assert ap.device_status(reset=True) == 5
    check_attention(q, kc, vc, bt, [L], True, 0.1, ap.attn_fwd_paged(*args))
    # a stage that no thread block gets to: nothing is withheld
    check_attention(q, kc, vc, bt, [L], True, 0.1,
                    ap.paged.fwd_paged_timeout_test(*args, drop_stage=10 ** 6))


# ---------------------------------------------------------------- what the status word says


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_a_timeout_is_not_hidden_by_a_bad_index(fmt):
    """Outputs are unspecified after a timeout, but not after an index out of range: where both
    happened, in whichever order and call, the status word says the first."""
    L, page, D = 3000, 16, 64
    bt, pages = tables([L], page, 111)
    kc, vc = (t.cuda() for t in pools(fmt, pages, 1, page, D, 112))
    q = randn(rng(113), 1, 4, 1, D).cuda()
    bad = bt.clone()
    bad[0, 0] = -1
    btd, badd, n = bt.cuda(), bad.cuda(), device_ints(L)
    k = randn(rng(114), 1, 1, 1, D).cuda()

    def append():
        ap.kv_append(k, k, kc, vc, badd, device_ints(0))

    def attend():
        ap.attn_fwd_paged(q, kc, vc, badd, n, True, 0.1)

    def give_up():
        ap.paged.fwd_paged_timeout_test(q, kc, vc, btd, n, True, 0.1, drop_stage=0,
                                        wait_budget_ns=20_000_000)

    for calls in ((append, give_up), (give_up, append), (attend, give_up), (give_up, attend),
                  (append, attend, give_up, append, attend)):
        for call in calls:
            call()
        torch.cuda.synchronize()
        assert ap.device_status(reset=False) == 5, [c.__name__ for c in calls]
        assert ap.device_status(reset=True) == 5
        assert ap.device_status(reset=True) == 0
    for call in (append, attend):
        call()
        torch.cuda.synchronize()
        assert ap.device_status(reset=True) == BAD_INDEX


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_counts_and_starts_out_of_range_are_recorded(fmt):
    """kv_append's new_lens below 0 or above S and kv_read's start beyond what the block table
    spans are cut, and the status word says so; at the range's ends it stays clean."""
    page, D, S, span = 16, 64, 3, 64
    bt, pages = tables([span, span], page, 115)
    kc, vc = (t.cuda() for t in pools(fmt, pages, 2, page, D, 116))
    k = randn(rng(117), 2, 2, S, D).cuda()
    start = device_ints(5, 30)

    def appended(*new):
        a, b = kc.clone(), vc.clone()
        ap.kv_append(k, k, a, b, bt.cuda(), start, new_lens=device_ints(*new))
        torch.cuda.synchronize()
        return a, b, ap.device_status(reset=True)

    for good, others in (((0, 3), ((-1, 3), (0, 4), (-2 ** 31, 2 ** 31 - 1))), ((3, 0), ((3, -5), (7, 0)))):
        want = appended(*good)
        assert want[2] == 0
        for new in others:
            got = appended(*new)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert got[2] == BAD_INDEX, new
    lens = device_ints(span, span)

    def read(*at):
        out = tuple(torch.full((2, 2, S, D), 3.0, dtype=torch.bfloat16).cuda() for _ in range(2))
        ap.kv_read(kc, vc, bt.cuda(), lens, S, start=device_ints(*at), out=out)
        torch.cuda.synchronize()
        return out, ap.device_status(reset=True)

    want, status = read(span - 1, span)
    assert status == 0 and (want[0][1] == 3.0).all() and (want[0][0, :, 1:] == 3.0).all()
    for at in ((span - 1, span + 1), (span - 1, 2 ** 31 - 1)):
        got, status = read(*at)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert status == BAD_INDEX, at
    got, status = read(-2 ** 31, 0)
    assert status == BAD_INDEX and (got[0][0] == 3.0).all() and not (got[0][1] == 3.0).any()


# ---------------------------------------------------------------- values of any size


@pytest.mark.parametrize("D,Hq,lens,wide", [
    (64, 1, [1, 2, 3, 17], False), (128, 4, [1, 300, 40], False), (128, 12, [5, 260], False),
    (64, 20, [33, 2], False), (128, 2, [5000, 3], True), (64, 3, [7000], True), (128, 40, [1300], True)])
@pytest.mark.parametrize("size", [3e38, 1e37, 2.0 ** 100, 2.0 ** -100, 2.0 ** -110])
def test_values_of_any_size_in_bf16(D, Hq, lens, wide, size):
    """Values next to the ends of bf16's range, of one sign and of both, under equal scores, scores
    that rise key by key and scores of a normal distribution: finite values give a finite O."""
    page, B = 16, len(lens)
    bt, pages = tables(lens, page, 121)
    if wide:
        bt = torch.cat([bt, torch.full((B, 80), -1, dtype=torch.int32)], 1)
    g = rng(122)
    k = randn(g, pages, 1, page, D)
    v = torch.full((pages, 1, page, D), size).to(torch.bfloat16)
    v[..., 1::2] *= (torch.randint(0, 2, (pages, 1, page, D // 2), generator=g) * 2 - 1).to(torch.bfloat16)
    q = randn(g, B, Hq, 1, D)
    rising = torch.zeros_like(k)
    for b, L in enumerate(lens):     # key x of the sequence: x / 16 in its first element
        for i in range(-(-L // page)):
            rising[int(bt[b, i]), 0, :, 0] = (torch.arange(page) + i * page) / 16.0
    q1 = torch.zeros_like(q)
    q1[..., 0] = 1.0
    for what, qq, kk, scale in (("equal", q, k, 0.0), ("rising", q1, rising, 1.0), ("normal", q, k, 0.2)):
        got = ap.attn_fwd_paged(qq.cuda(), kk.cuda(), v.cuda(), bt.cuda(), device_ints(*lens), True, scale)
        check_attention(qq, kk, v, bt, lens, True, scale, got, what=(what, size))


@pytest.mark.parametrize("size", [2.0 ** 30, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("fmt,D,Hq", [("int4", 64, 4), ("int4", 128, 2), ("int4", 128, 12), ("bf16", 128, 2),
                                      ("bf16", 64, 12)])
def test_a_large_value_that_a_row_does_not_see_does_not_matter(fmt, D, Hq, size):
    """The last token's value is finite and far larger than the others: of four causal queries only
    the last one sees it, and the others' results are as exact as without it."""
    for L in (4, 45, 1300):
        page = 16
        bt, pages = tables([L], page, 131)
        bt = torch.cat([bt, torch.full((1, 2), -1, dtype=torch.int32)], 1)
        g = rng(132)
        k, v = randn(g, pages, 1, page, D), randn(g, pages, 1, page, D)
        kc, small = fill(k, fmt, "k"), fill(v, fmt, "v")
        pg, slot = int(bt[0, (L - 1) // page]), (L - 1) % page
        v[pg, 0, slot] *= size
        vc = fill(v, fmt, "v")
        q = randn(g, 1, Hq, 4, D)
        o, lse = ap.attn_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), bt.cuda(), device_ints(L), True, 0.1)
        head = (o[:, :, :3].contiguous(), lse[:, :, :3].contiguous())
        check_attention(q[:, :, :3], kc, small, bt, [L - 1], True, 0.1, head, what=L)
        check_attention(q, kc, vc, bt, [L], True, 0.1, (o, lse), what=L)


# ---------------------------------------------------------------- many short items


def short_lens(B, seed, most=1024):
    """Mostly short, some empty, a few as long as the block table."""
    g = np.random.default_rng(seed)
    n = [int(x) for x in np.exp(g.uniform(0, np.log(130), B))]
    n[0], n[B // 3], n[B // 2], n[-1] = 0, most, 1000, 0
    return n


@pytest.mark.parametrize("fmt,D,B,H,group,Sq,causal", [
    ("int4", 128, 40, 4, 2, 1, True), ("bf16", 128, 40, 4, 2, 1, True),
    ("int4", 64, 150, 4, 1, 2, True), ("bf16", 64, 150, 4, 1, 2, False),
    ("int4", 128, 300, 3, 1, 1, False), ("bf16", 128, 300, 3, 2, 1, True),
    ("int4", 64, 160, 1, 8, 1, True), ("bf16", 64, 1300, 1, 1, 1, True),
    ("int4", 64, 140, 2, 5, 3, True), ("bf16", 128, 140, 2, 5, 3, True)])
def test_many_short_items(fmt, D, B, H, group, Sq, causal):
    """Block tables of at most 1024 keys (items kept whole) and more items than SMs, up to several
    for every thread block, lengths from 0 on: each block walks its items in turn, with more
    sequences than the plan has threads."""
    page = 64
    lens = short_lens(B, 141)
    bt, pages = tables([max(n, 1) for n in lens], page, 142)
    assert bt.shape[1] * page == 1024
    kc, vc = pools(fmt, pages, H, page, D, 143)
    q = randn(rng(144), B, H * group, Sq, D)
    q_lens = [(3 * b) % (Sq + 1) for b in range(B)] if Sq > 1 else None
    out = (torch.full((B, H * group, Sq, D), 5.0, dtype=torch.bfloat16).cuda(),
           torch.full((B, H * group, Sq), 5.0).cuda())
    ap.attn_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), bt.cuda(), device_ints(*lens), causal, 0.11,
                      q_lens=device_ints(*q_lens) if q_lens else None, out=out)
    torch.cuda.synchronize()
    check_attention(q, kc, vc, bt, lens, causal, 0.11, out, q_lens)
    for b in range(B if q_lens else 0):
        assert (out[0][b, :, q_lens[b]:] == 5.0).all() and (out[1][b, :, q_lens[b]:] == 5.0).all()


# ---------------------------------------------------------------- bytes that only a 4-bit cache has


def packed_tokens(x, kind, page):
    """Values [1, H, L, D] (bf16, L a multiple of 16) as the 4-bit blocks [L / page, H, page / 16, 9 D]
    of pages in order."""
    _, H, L, D = x.shape
    b = ref.pack(ref.f64(x).reshape(-1, D), kind)
    return torch.from_numpy(b).reshape(H, L // page, page // 16, 9 * D).transpose(0, 1)


def test_a_4_bit_pool_larger_than_32_bit_offsets():
    """The appended bytes lie in the last pages of a pool of more than 2^32 bytes, and nowhere else
    in the pages that an offset cut to 32 bits would reach; they are read back from there."""
    H, page, D, L = 8, 64, 128, 256
    per = H * page * 72
    pages = (1 << 32) // per + 40
    kc, vc = ap.kv_cache_empty(pages, H, page, D, "int4")
    kc.fill_(0x5a), vc.fill_(0x5a)
    bt = torch.arange(pages - 1, pages - 5, -1, dtype=torch.int32)[None].cuda()
    k, v = (randn(rng(151 + i), 1, H, L, D) for i in range(2))
    ap.kv_append(k.cuda(), v.cuda(), kc, vc, bt, device_ints(0))
    got = ap.kv_read(kc, vc, bt, device_ints(L), L)
    torch.cuda.synchronize()
    for pool, x, kind, back in ((kc, k, "k", got[0]), (vc, v, "v", got[1])):
        want = packed_tokens(x, kind, page)
        assert torch.equal(pool[pages - 4:].flip(0).cpu(), want)
        assert (pool[:48] == 0x5a).all() and (pool[pages - 8:pages - 4] == 0x5a).all()
        vals = ref.unpack(want.transpose(0, 1).reshape(-1, 9 * D).numpy(), kind)[0]
        assert np.array_equal(ref.f64(back), ref.bf16(vals).reshape(1, H, L, D))


def test_scales_and_keys_of_every_ratio():
    """The groups of test_quantisation_of_every_ratio, and others down to bf16's smallest numbers:
    the scales' bytes, and the codes of keys as well as of values."""
    D = 64
    m = np.arange(128, 256) / 128.0
    tops = np.concatenate([m * 2.0 ** e for e in (0, 1, -1, 37, -98, -99, -120, -125, -126, -128, -131, -133, 127)])
    tops = torch.from_numpy(tops).to(torch.bfloat16).double().numpy()
    g = np.random.default_rng(153)
    x = g.uniform(-1, 1, (len(tops), 32)) * tops[:, None]
    x[np.arange(len(tops)), g.integers(0, 32, len(tops))] = tops * np.where(g.random(len(tops)) < 0.5, -1, 1)
    x = torch.from_numpy(x.reshape(-1, D)).to(torch.bfloat16)
    S = len(x)
    kc, vc = ap.kv_cache_empty(-(-S // 64), 1, 64, D, "int4")
    kc.zero_(), vc.zero_()
    bt = torch.arange(kc.shape[0], dtype=torch.int32)[None].cuda()
    xd = x[None, None].cuda()
    ap.kv_append(xd, xd, kc, vc, bt, device_ints(0))
    back = ap.kv_read(kc, vc, bt, device_ints(S), S)
    torch.cuda.synchronize()
    f = x.double().numpy().reshape(S, D // 32, 32)
    scale = torch.from_numpy(np.abs(f).max(-1) / 7).to(torch.bfloat16)   # (subnormals too)
    s = scale.double().numpy()[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s > 0, np.clip(np.round(f / s), -7, 7), 0)
    code = (c + 8).astype(np.uint8).reshape(S, D)
    bytes_of = scale.view(torch.int16).numpy().view(np.uint8).reshape(S, D // 16)
    want_back = torch.from_numpy((c * s).reshape(S, D)).to(torch.bfloat16)
    for pool, kind, b in ((kc, "k", back[0]), (vc, "v", back[1])):
        got = pool.cpu().numpy().reshape(-1, 9 * D)
        idx = ref.nibble_index(kind, D)
        for t in range(S):
            blk, r = got[t // 16], t % 16
            assert np.array_equal((blk[idx[r] // 2] >> (4 * (idx[r] % 2))) & 15, code[t]), (kind, t)
            at = 8 * D + r * (D // 16)
            assert np.array_equal(blk[at:at + D // 16], bytes_of[t]), (kind, t)
        assert np.array_equal(ref.f64(b[0, 0]), want_back.double().numpy())


# ---------------------------------------------------------------- queries rotated in place


@pytest.mark.parametrize("fmt,D,S,rot,inter", [
    ("int4", 128, 1, 128, False), ("int4", 64, 33, 32, True), ("bf16", 128, 40, 64, False),
    ("bf16", 64, 1, 64, True), ("int4", 128, 700, 128, False), ("bf16", 128, 9, 16, False)])
def test_queries_rotated_in_place(fmt, D, S, rot, inter):
    """q_out may be q itself: the same bits as into another tensor, padding untouched."""
    B, Hq, H, page = 2, 12, 2, 32
    new = [S, S // 2]
    bt, pages = tables([S + 7] * B, page, 161)
    cos, sin = (t.cuda() for t in rope(S + 7, rot))
    g = rng(162)
    q, k, v = (randn(g, B, h, S, D).cuda() for h in (Hq, H, H))
    pool = [[t.cuda() for t in pools(fmt, pages, H, page, D, 163)] for _ in range(2)]
    args = (bt.cuda(), device_ints(0, 7))
    kw = dict(cos=cos, sin=sin, new_lens=device_ints(*new), interleaved=inter)
    want = ap.kv_append(k, v, *pool[0], *args, q=q, q_out=q.clone(), **kw)
    got = q.clone()
    assert ap.kv_append(k, v, *pool[1], *args, q=got, q_out=got, **kw) is got
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got[1, :, new[1]:], q[1, :, new[1]:])
    assert S == 1 or not torch.equal(got[0], q[0])       # (position 0 turns by nothing)
    for a, b in zip(*pool):
        assert torch.equal(a, b)


def test_more_tokens_than_an_int_are_refused():
    """A view of one token that claims 2^32 + 1 of them: its length must not be cut to 32 bits."""
    D = 64
    kc, vc = ap.kv_cache_empty(1, 1, 16, D)
    kc.zero_(), vc.zero_()
    bt = torch.zeros((1, 1), dtype=torch.int32).cuda()
    one = torch.ones((1, 1, 1, D), dtype=torch.bfloat16).cuda()
    for n in (2 ** 32 + 1, 2 ** 31):
        many = one.expand(1, 1, n, D)
        with pytest.raises((ap.AttnError, ValueError)):
            ap.kv_append(many, many, kc, vc, bt, device_ints(0), new_lens=device_ints(1))
    torch.cuda.synchronize()
    assert (kc == 0).all() and (vc == 0).all()


def test_without_torch_s_short_ways(monkeypatch):
    """The same bits by way of torch.cuda's public functions, on the current and on another stream,
    with the workspace that the call allocates freed again."""
    D, H, page, L = 64, 2, 32, 4000
    bt, pages = tables([L], page, 181)
    kc, vc = (t.cuda() for t in pools("int4", pages, H, page, D, 182))
    btd, n, q = bt.cuda(), device_ints(L), randn(rng(183), 1, 8, 1, D).cuda()
    want = ap.attn_fwd_paged(q, kc, vc, btd, n, True, 0.1)
    out = (torch.zeros_like(want[0]), torch.zeros_like(want[1]))
    ways = ap.paged._short_ways(object())
    for name, way in zip(("_current_device", "_current_stream", "_alloc", "_free"), ways):
        monkeypatch.setattr(ap.paged, name, way)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for stream in (None, torch.cuda.Stream()):
        out[0].zero_(), out[1].zero_()
        torch.cuda.synchronize()
        ap.attn_fwd_paged(q, kc, vc, btd, n, True, 0.1, out=out, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert torch.cuda.memory_allocated() == before


# ---------------------------------------------------------------- how exact a bf16 cache's attention is


@pytest.mark.parametrize("D,group,Sq,lens,wide", [
    (128, 4, 1, [500, 37], False), (64, 1, 1, [1000], False), (128, 8, 1, [90, 400], False),
    (64, 2, 3, [300, 6], False), (128, 4, 1, [6000], True), (64, 1, 8, [2000], True)])
def test_probabilities_of_up_to_eight_rows_keep_sixteen_bits(D, group, Sq, lens, wide):
    """With up to eight query rows a KV head the second product takes a probability as the sum of two
    bf16 numbers: off by half a step of the second, 2^-16 of it.  The bound of O is that of the reference with this share in place of
    one bf16 number's 2^-8, and exponents of up to 32, of which a subtraction's rounding is 2^-20."""
    page, B, scale = 64, len(lens), 0.1
    bt, pages = tables(lens, page, 171)
    if wide:
        bt = torch.cat([bt, torch.full((B, 20), -1, dtype=torch.int32)], 1)
    kc, vc = pools("bf16", pages, 1, page, D, 172)
    q = randn(rng(173), B, group, Sq, D)
    o, _ = ap.attn_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), bt.cuda(), device_ints(*lens), True, scale)
    o, kv, vv, qf = ref.f64(o), ref.f64(kc), ref.f64(vc), ref.f64(q)
    for b, L in enumerate(lens):
        k, v = ref.gather(kv, bt[b].numpy(), L, page)[0], ref.gather(vv, bt[b].numpy(), L, page)[0]
        for h in range(group):
            for i in range(Sq):
                n = max(0, L - Sq + i + 1)
                x = qf[b, h, i]
                s = scale * (k[:n] @ x)
                p = np.exp(s - s.max())
                want, A = p @ v[:n] / p.sum(), p @ np.abs(v[:n]) / p.sum()
                e = (scale * (np.abs(k[:n]) @ np.abs(x))).max() * 2.0 ** -18 + np.abs(s).max() * 1.5 * 2.0 ** -22 \
                    + 2.0 ** -20 + 2.0 ** -22
                tol = 1.01 * (2.0 ** -16 + 2 * e) * A
                tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
                assert (np.abs(o[b, h, i] - want) <= tol).all(), (b, h, i, (np.abs(o[b, h, i] - want) / tol).max())


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_prompts_behind_cached_prefixes_in_two_parts(fmt):
    """attn_fwd's causal mask begins at its first key, so a prompt behind a cached prefix is two of
    its calls, joined by their log-sum-exps: the prefix as kv_read returns it without mask, the new
    tokens' keys with.  Against attn_fwd_paged's 64-bit reference: each part's O is rounded to bf16
    (2^-8) and has probabilities rounded to bf16 (2^-8 of A, the sum of |shares|), which the
    reference's bound has once, and its scores are in fp32 as the reference's bound takes them;
    kv_read rounds 4-bit values to bf16, 2^-8 of a value and, through the keys, of a score's terms."""
    D, Hq, H, page, scale = 64, 4, 2, 32, 0.125
    for prefix, new in ((37, 20), (300, 129), (64, 1)):
        L = prefix + new
        bt, pages = tables([L], page, 191)
        kc, vc = pools(fmt, pages, H, page, D, 192)
        q = randn(rng(193), 1, Hq, new, D)
        n = device_ints(L)
        kd, vd, bd, qd = kc.cuda(), vc.cuda(), bt.cuda(), q.cuda()
        k, v = ap.kv_read(kd, vd, bd, n, prefix)
        k2, v2 = ap.kv_read(kd, vd, bd, n, new, start=device_ints(prefix))
        parts = [ap.attn_fwd(qd, k, v, False, scale), ap.attn_fwd(qd, k2, v2, True, scale)]
        lse = torch.logaddexp(parts[0][1], parts[1][1])
        o = sum(p[0].float() * torch.exp(p[1] - lse)[..., None] for p in parts)
        kv, ks = ref.cache_values(kc, "k")
        vv, vs = ref.cache_values(vc, "v")
        args = bt.numpy(), [L], page, True, scale
        ro, rl, _, _ = ref.attention(ref.f64(q), kv, vv, ks, vs, *args)
        ra = ref.attention(ref.f64(q), kv, np.abs(vv), ks, vs, *args)[0]     # A
        es = scale * max(np.abs(kv[:, h // 2]).reshape(-1, D).max(0) @ np.abs(ref.f64(q[0, h])).max(0)
                         for h in range(Hq))
        e = es * (2.0 ** -18 + (2.0 ** -8 if fmt == "int4" else 0)) + 2.0 ** -19
        tol = (2.0 ** -8 * (2 if fmt == "bf16" else 3) + 2 * e) * 1.02 * ra
        assert (np.abs(ref.f64(o) - ro) <= tol).all()
        assert np.abs(ref.f64(lse) - rl).max() <= e + 2.0 ** -8
        got = ap.attn_fwd_paged(qd, kd, vd, bd, n, True, scale)
        check_attention(q, kc, vc, bt, [L], True, scale, got)
