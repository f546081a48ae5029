"""The entry points of packed sequences refuse bad arguments on the host, before any CUDA call
(CPU only; fake, never-dereferenced device addresses), and the reference of the GPU tests holds
against torch's own arithmetic and against differences."""
import ctypes
import math
import struct
import subprocess

import pytest
import torch

import attention_pipelining_gb300 as ap
from attention_pipelining_gb300 import _build, packed
from tests import packed_ref as ref

A = 0x10000
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    ap.build()
    return ap._load()


def sizes(**kw):
    d = dict(B=2, T_q=100, T_k=100, H_q=8, H_kv=2, D=128, causal=1, scale=0.1)
    d.update(kw)
    return packed._SIZES.pack(*[d[n] for n in ("B", "T_q", "T_k", "H_q", "H_kv", "D", "causal", "scale")])


def thd(data=A, st=12 * 128, sh=128):
    return packed._THD.pack(data or 0, st, sh)


def fwd(lib, s=None, q=None, k=None, v=None, o=None, lse=A, cu_q=A, cu_k=A, ws=A, nbytes=BIG):
    return lib.attn_fwd_packed(sizes() if s is None else s, q or thd(), k or thd(), v or thd(), o or thd(),
                               lse, cu_q, cu_k, ws, nbytes, None)


def bwd(lib, s=None, lse=A, cu_q=A, cu_k=A, ws=A, nbytes=BIG, det=0, **kw):
    t = [kw.get(n) or thd() for n in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")]
    return lib.attn_bwd_packed(sizes() if s is None else s, *t[:4], lse, *t[4:], cu_q, cu_k, ws, nbytes, det,
                               None)


def rope(lib, q=True, qo=True, k=True, ko=True, positions=A, sections=(16, 24, 24), axes=None, cos=A, sin=A,
         rows=512, rot=128, inter=0, inverse=0, T=10, H_q=8, H_kv=2, D=128):
    t = [thd() if x is True else x for x in (q, qo, k, ko)]
    sec = None if sections is None else struct.pack(f"@{len(sections)}i", *sections)
    return lib.attn_rope_packed(*t, positions, sec, len(sections or ()) if axes is None else axes, cos, sin,
                                rows, rot, inter, inverse, T, H_q, H_kv, D, None)


BAD_SIZES = [(dict(B=0), 1), (dict(T_q=0), 1), (dict(T_k=-1), 1), (dict(H_q=0), 1), (dict(H_kv=0), 1),
             (dict(H_q=9), 1), (dict(D=0), 1), (dict(causal=2), 1), (dict(scale=math.nan), 1),
             (dict(scale=math.inf), 1), (dict(D=96), 2), (dict(B=70000), 2), (dict(H_q=70000, H_kv=70000), 2), (dict(H_q=33, H_kv=1), 2),
             (dict(H_q=132, H_kv=1), 2), (dict(H_q=127, H_kv=1), 2), (dict(T_q=1 << 30), 2),
             (dict(T_k=1 << 30), 2), (dict(T_k=(1 << 30) - 1, H_q=60000, H_kv=60000), 2),
             (dict(T_q=(1 << 30) - 1, H_q=128, H_kv=128), 2)]


@pytest.mark.parametrize("kw,code", BAD_SIZES, ids=[str(k) for k, _ in BAD_SIZES])
def test_sizes_are_checked(lib, kw, code):
    s = sizes(**kw)
    assert fwd(lib, s) == code
    assert bwd(lib, s) == code
    assert lib.attn_packed_workspace_bytes(s) == 0
    assert lib.attn_packed_bwd_workspace_bytes(s, 0) == 0


def test_no_sizes(lib):
    assert lib.attn_fwd_packed(None, thd(), thd(), thd(), thd(), A, A, A, A, BIG, None) == 1
    assert lib.attn_packed_workspace_bytes(None) == 0


BAD_TENSOR = [(dict(data=None), 1), (dict(data=A + 8), 3), (dict(st=12 * 128 + 4), 3), (dict(sh=12), 3),
              (dict(st=0), 2), (dict(st=-1536), 2), (dict(sh=-128), 2), (dict(sh=0), 2), (dict(st=1 << 40), 2)]


@pytest.mark.parametrize("kw,code", BAD_TENSOR, ids=[str(k) for k, _ in BAD_TENSOR])
def test_tensors_are_checked(lib, kw, code):
    for n in ("q", "k", "v", "o"):
        assert fwd(lib, **{n: thd(**kw)}) == code, n
    for n in ("q", "k", "v", "o", "dout", "dq", "dk", "dv"):
        assert bwd(lib, **{n: thd(**kw)}) == code, n
    for n in ("q", "qo", "k", "ko"):
        assert rope(lib, **{n: thd(**kw)}) == code, n


def test_strides_of_single_dimensions_are_not_looked_at(lib):
    odd = thd(sh=3, st=-5)
    s = sizes(T_q=1, T_k=1, H_q=1, H_kv=1)
    assert fwd(lib, s, q=odd, k=odd, v=odd, o=odd, lse=A + 2) == 3      # stops at lse's address
    assert bwd(lib, s, q=odd, k=odd, v=odd, o=odd, dout=odd, dq=odd, dk=odd, dv=odd, lse=None) == 1
    assert rope(lib, q=odd, qo=odd, k=odd, ko=odd, T=1, H_q=1, H_kv=1, cos=A + 8) == 3


@pytest.mark.parametrize("kw,code", [
    (dict(lse=None), 1), (dict(lse=A + 2), 3), (dict(cu_q=None), 1), (dict(cu_q=A + 1), 3),
    (dict(cu_k=A + 2), 3), (dict(ws=None), 1), (dict(ws=A + 16), 3), (dict(nbytes=100), 1)])
def test_attention_refuses(lib, kw, code):
    assert fwd(lib, **kw) == code
    assert bwd(lib, **kw) == code


@pytest.mark.parametrize("drop,budget", [(-1, 10**7), (0, 999_999), (0, 2**63)])
def test_timeout_hooks_refuse(lib, drop, budget):
    t = [thd() for _ in range(8)]
    assert lib.attn_fwd_packed_timeout_test(sizes(), *t[:4], A, A, A, A, BIG, drop, budget, None) == 1
    assert lib.attn_bwd_packed_timeout_test(sizes(), *t[:4], A, *t[4:], A, A, A, BIG, 0, drop, budget, None) == 1


def test_more_refusals(lib):
    assert bwd(lib, det=2) == 1
    assert fwd(lib, sizes(T_k=200), cu_k=None) == 1        # other keys, without their bounds
    assert bwd(lib, sizes(T_k=200), cu_k=None) == 1
    need = lib.attn_packed_workspace_bytes(sizes())
    assert fwd(lib, nbytes=need - 1) == 1
    assert fwd(lib, nbytes=need, cu_q=A + 2) == 3          # stops at another rule
    for det in (0, 1):
        need = lib.attn_packed_bwd_workspace_bytes(sizes(), det)
        assert bwd(lib, nbytes=need - 1, det=det) == 1
        assert bwd(lib, nbytes=need, det=det, cu_q=A + 2) == 3
    assert lib.attn_packed_bwd_workspace_bytes(sizes(), 2) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), 1), (dict(H_q=-1), 1), (dict(H_q=0), 1), (dict(q=None), 1), (dict(qo=None), 1),
    (dict(ko=None), 1), (dict(H_kv=0), 1), (dict(H_q=0, H_kv=0, q=None, qo=None, k=None, ko=None), 1),
    (dict(positions=None), 1), (dict(sections=None), 1), (dict(sections=(64, 0)), 1),
    (dict(sections=(64, -1, 1)), 1), (dict(sections=(63,)), 1), (dict(sections=(13,) * 4 + (12,), axes=5), 1),
    (dict(sections=(2 ** 31 - 1, 2 ** 31 - 1, 66, 64)), 1), (dict(axes=0), 1), (dict(rot=144), 1),
    (dict(rot=120, sections=(60,)), 1), (dict(rot=0), 1), (dict(rows=0), 1), (dict(inter=2), 1),
    (dict(inverse=-1), 1), (dict(cos=None), 1), (dict(sin=None), 1), (dict(D=96, rot=96, sections=(48,)), 2),
    (dict(D=256), 2), (dict(T=1 << 30), 2), (dict(H_q=40000), 2), (dict(positions=A + 2), 3), (dict(cos=A + 8), 3),
    (dict(sin=A + 4), 3)])
def test_rotation_refuses(lib, kw, code):
    assert rope(lib, **kw) == code


def test_workspace_holds_the_lists(lib):
    """A header, the bounds, 48 and 64 bytes for each tile and key block that there may be, with up to 4/3
    of 152 parts, a part's results where any entry can be cut (12 blocks of keys, 3 tiles), two counters a part, and (backward)
    two row vectors and the accumulator."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for H_q, H_kv, positions in ((8, 8, 128), (8, 2, 32), (6, 2, 40), (5, 1, 24), (7, 1, 16), (32, 1, 4),
                                 (31, 1, 4), (128, 1, 1), (40, 1, 3), (512, 256, 64)):
        R = H_q // H_kv
        for B, T in ((1, 1), (3, 1000), (3, 1500), (500, 77)):
            s = sizes(B=B, T_q=T, T_k=T + 3, H_q=H_q, H_kv=H_kv, D=64)
            slots = 4 * 152 // (3 * H_kv)
            counters = up(slots * H_kv * 2 * 4)
            begin = 256 + 2 * up(4 * (B + 1)) + up(8 * (B + 1))
            tiles = up(48 * (T // (2 * positions) + B + slots)) + counters
            if -(-(T + 3) // 128) >= 12:
                tiles += up(slots * H_kv * 256 * 64 * 4)
                lse = up(slots * H_kv * 256 * 4)
            else:
                lse = 0
            assert lib.attn_packed_workspace_bytes(s) == begin + tiles + lse
            blocks = (T + 3) // 128 + B + slots
            keys = up(64 * blocks) + up(4 * blocks) + counters
            if -(-T // positions) >= 3:
                keys += up(slots * H_kv * 256 * 64 * 4)
            vec = (T + 4 * B + 4) * R + 128
            vec += -vec % 4
            keys += 2 * up(4 * H_kv * vec)
            assert lib.attn_packed_bwd_workspace_bytes(s, 1) == begin + tiles + keys
            assert lib.attn_packed_bwd_workspace_bytes(s, 0) == begin + keys + up(4 * T * H_q * 64)


# the least blocks of keys (forward, dq) or query tiles (dk, dv) that are cut into parts: one and a half
# times a part's least
CUT_KEYS = 12
CUT_TILES = {64: 3, 128: 5}


@pytest.mark.parametrize("D", [64, 128])
def test_where_work_may_be_cut(lib, D):
    """The workspace has room for parts' results from these numbers on (test_around_the_least_parts has
    works of just that many blocks)."""
    def grows(nbytes, field, blocks, step):
        """What the last token that makes it so many blocks adds, beside what each token takes"""
        at = (blocks - 1) * step
        a, b, c = (nbytes(sizes(B=1, H_q=1, H_kv=1, D=D, **{**dict(T_q=5, T_k=5), field: at + n})) for n in (-1, 0, 1))
        return c - b - (b - a)

    slots = 4 * 152 // 3
    tile, keys = slots * 256 * D * 4, slots * 2 * 128 * D * 4
    fwd = lib.attn_packed_workspace_bytes
    assert grows(fwd, "T_k", CUT_KEYS - 1, 128) < 1000
    assert grows(fwd, "T_k", CUT_KEYS, 128) >= tile
    for det in (0, 1):
        bwd = lambda s: lib.attn_packed_bwd_workspace_bytes(s, det)  # noqa: E731
        assert grows(bwd, "T_q", CUT_TILES[D] - 1, 128) < 2000
        assert grows(bwd, "T_q", CUT_TILES[D], 128) >= keys - 2000
        assert grows(bwd, "T_k", CUT_KEYS - 1, 128) < 2000
        assert (grows(bwd, "T_k", CUT_KEYS, 128) >= tile) == bool(det)


# query heads a key head that the calls take
GROUPS = [g for g in range(1, 129) if g <= 32 or g % 4 == 0]


def test_boxes_of_o_hold_rows_of_their_tile_alone(lib):
    """Where O leaves by boxes of 32 rows, each box is those rows in their order and none of them is a
    spare one, which would be a row of the next token; and all rows that could leave so do."""
    for R in GROUPS:
        rows = R * (128 // R if R % 4 == 0 else 32 // R * 4)
        boxes = lib.attn_fwd_packed_o_boxes(sizes(H_q=3 * R, H_kv=3))
        heads, could = min(R, 32), 0
        for i in range(4):
            t0, h0 = 32 * i // R, 32 * i % R
            box = [(t0 + t) * R + h0 + h for t in range(32 // heads) for h in range(heads)]
            if h0 + heads <= R and box == list(range(32 * i, 32 * i + 32)) and box[-1] < rows and could == i:
                could += 1
        if R % 32 and 32 % R:
            could = 0   # (a box's shape would change from row to row)
        assert boxes == could, (R, boxes, could)
    assert lib.attn_fwd_packed_o_boxes(sizes(H_q=33, H_kv=1)) == -1
    assert lib.attn_fwd_packed_o_boxes(None) == -1


DIVISIONS = r"""
#include <cstdio>
#include "attn_internal.h"
int main() {
  for (long long d = 1; d <= 256; ++d) {
    const unsigned long long inverse = ((1ull << 40) + d - 1) / d;
    const long long most = (1ll << 31) - 1;
    for (int bit = 0; bit <= 31; ++bit)
      for (long long around : {1ll << bit, (1ll << bit) * d, (most >> bit) / d * d})
        for (long long x = around - 2; x <= around + 2; ++x)
          if (x >= 0 && x <= most && attnpipe::packed_over((int)x, inverse) != x / d) {
            std::printf("%lld / %lld gave %d\n", x, d, attnpipe::packed_over((int)x, inverse));
            return 1;
          }
  }
  return 0;
}
"""


def test_divisions_by_an_inverse(tmp_path):
    """packed_over over the whole range that the sizes admit: around powers of two, alone and times the
    divisor, and around the largest multiples."""
    src, exe = tmp_path / "over.cpp", tmp_path / "over"
    src.write_text(DIVISIONS)
    subprocess.run([_build.nvcc(), "-std=c++17", "-O1", "-I", _build.INCLUDE, "-I", _build.CSRC, str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_binding_refuses_on_the_host():
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    f = torch.zeros(8, 32)
    for call in (lambda: ap.attn_fwd_packed(t, t, t, cu, True, 0.1),
                 lambda: ap.attn_bwd_packed(t, t, t, t, f, t, cu, True, 0.1),
                 lambda: ap.rope_packed(t, t, cu[None], f, f),
                 lambda: ap.rope_packed(None, None, cu[None], f, f)):
        with pytest.raises(TypeError):   # not on a GPU, or no tensor at all
            call()


@pytest.fixture
def on_the_host(lib, monkeypatch):
    """The binding's checks, with tensors on the host in place of a GPU's (they stop before any launch)."""
    packed._import()
    monkeypatch.setattr(packed, "_device", lambda name, t: t.get_device())


@pytest.mark.parametrize("H_q,H_kv,D,scale,code", [
    (33, 1, 64, 0.1, 2), (132, 1, 64, 0.1, 2), (2, 2, 96, 0.1, 2), (2, 2, 32, 0.1, 2), (3, 2, 64, 0.1, 1),
    (2, 2, 64, math.nan, 1), (2, 2, 64, -math.inf, 1)])
def test_binding_says_why_it_refuses_sizes(on_the_host, H_q, H_kv, D, scale, code):
    """The status is the C entry's: what is not supported is no invalid argument."""
    q, k = (torch.zeros(4, h, D, dtype=torch.bfloat16) for h in (H_q, H_kv))
    cu, lse = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(H_q, 4)
    for call in (lambda: ap.attn_fwd_packed(q, k, k, cu, True, scale),
                 lambda: ap.attn_bwd_packed(q, k, k, q, lse, q, cu, True, scale),
                 lambda: ap.attn_bwd_packed(q, k, k, q, lse, q, cu, True, scale, deterministic=True)):
        with pytest.raises(ap.AttnError) as e:
            call()
        assert e.value.code == code, e.value


@pytest.mark.parametrize("which", ["q", "k", "T_q"])
def test_binding_refuses_sizes_beyond_its_ints(on_the_host, which):
    """Views that claim 2^31 heads or tokens."""
    n = 2 ** 31
    q, k = torch.zeros(4, 1, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    if which == "q":
        q = q.expand(4, n, 64)
    elif which == "k":
        k = k.expand(4, n, 64)
    else:
        q = q[:1].expand(n, 1, 64)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="below 2\\^31"):
        ap.attn_fwd_packed(q, k, k, cu, True, 0.1, cu_k=cu)
    with pytest.raises(ValueError, match="below 2\\^31"):
        ap.attn_bwd_packed(q, k, k, q, torch.zeros(1, 4), q, cu, True, 0.1, cu_k=cu)


def test_a_stream_of_another_device_is_refused(on_the_host):
    """With a text that names what the call has: tensors, no cache."""
    class Stream:
        device = torch.device("cuda", 5)

    q = torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    cu, table = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(8, 32)
    for call in (lambda: ap.attn_fwd_packed(q, q, q, cu, True, 0.1, stream=Stream),
                 lambda: ap.attn_bwd_packed(q, q, q, q, torch.zeros(1, 4), q, cu, True, 0.1, stream=Stream),
                 lambda: ap.rope_packed(q, q, cu[None, :1].expand(1, 4).contiguous(), table, table, stream=Stream)):
        with pytest.raises(ValueError, match="stream belongs to another device than the tensors"):
            call()


# ---------------------------------------------------------------- the reference itself

CASES = [([5, 0, 3], [5, 0, 3], True), ([4, 2], [6, 1], True), ([3, 0, 2], [4, 3, 0], False)]


def data(lens_q, lens_k, H_q=4, H_kv=2, D=8, seed=0):
    g = torch.Generator().manual_seed(seed)
    cu_q, cu_k = ref.bounds(lens_q), ref.bounds(lens_k)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return (r(cu_q[-1], H_q, D), r(cu_k[-1], H_kv, D), r(cu_k[-1], H_kv, D), r(cu_q[-1], H_q, D), cu_q, cu_k)


@pytest.mark.parametrize("lens_q,lens_k,causal", CASES)
def test_reference_forward(lens_q, lens_k, causal):
    """Row by row with softmax and logsumexp of torch."""
    q, k, v, _, cu_q, cu_k = data(lens_q, lens_k)
    o, lse, to, tl = ref.forward(q, k, v, cu_q, cu_k, causal, 0.3)
    for b, (n, m) in enumerate(zip(lens_q, lens_k)):
        for i in range(n):
            see = max(0, min(m, i + m - n + 1)) if causal else m
            for h in range(4):
                t = cu_q[b] + i
                kk, vv = (x[cu_k[b]:cu_k[b] + see, h // 2] for x in (k, v))
                if see == 0:
                    assert (o[t, h] == 0).all() and lse[h, t] == -math.inf
                    continue
                s = 0.3 * kk @ q[t, h]
                assert torch.allclose(torch.softmax(s, 0) @ vv, o[t, h], atol=1e-12)
                assert torch.allclose(torch.logsumexp(s, 0), lse[h, t], atol=1e-12)
    assert (to[torch.isfinite(o)] >= 0).all() and (tl[torch.isfinite(lse)] >= 0).all()


@pytest.mark.parametrize("lens_q,lens_k,causal", CASES)
def test_reference_backward_against_differences(lens_q, lens_k, causal):
    q, k, v, do, cu_q, cu_k = data(lens_q, lens_k)
    o, lse, _, _ = ref.forward(q, k, v, cu_q, cu_k, causal, 0.3)
    got = ref.backward(q, k, v, o, lse, do, cu_q, cu_k, causal, 0.3)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        flat = x.view(-1)
        for i in range(0, flat.numel(), 3):
            was, h, ends = flat[i].item(), 1e-5, []
            for d in (h, -h):
                flat[i] = was + d
                ends.append((ref.forward(q, k, v, cu_q, cu_k, causal, 0.3)[0] * do).sum().item())
            flat[i] = was
            d = (ends[0] - ends[1]) / (2 * h)
            # central differences: h^2 times the third derivative, and 2^-52 / h of the sum's rounding
            assert abs(d - got[name][0].view(-1)[i].item()) <= 1e-7 * (1 + abs(d)), (name, i)


def test_reference_rotation():
    """One axis against complex numbers; several axes section by section; the inverse undoes it to
    within the two roundings."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 3, 32, generator=g).bfloat16().double()
    pos = torch.randint(0, 50, (3, 6), generator=g)
    ang = torch.arange(50)[:, None] * 0.3 ** torch.arange(16)
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    y = ref.rope(x, pos[:1], cos, sin, [16], True, False)
    z = torch.view_as_complex(x.view(6, 3, 16, 2).contiguous()) * torch.complex(cos, sin)[pos[0]][:, None].to(torch.complex128)
    assert torch.equal(y, ref.round_bf16(torch.view_as_real(z).flatten(2)))
    y = ref.rope(x, pos, cos, sin, [3, 8, 5], False, False)
    for a, lo, hi in ((0, 0, 3), (1, 3, 11), (2, 11, 16)):
        one = ref.rope(x, pos[a:a + 1], cos, sin, [16], False, False)
        assert torch.equal(y[..., lo:hi], one[..., lo:hi]) and torch.equal(y[..., 16 + lo:16 + hi], one[..., 16 + lo:16 + hi])
    back = ref.rope(y, pos, cos, sin, [3, 8, 5], False, True)
    r = (x[..., :16] ** 2 + x[..., 16:] ** 2).sqrt().repeat(1, 1, 2)
    assert ((back - x).abs() <= 3 * 2.0 ** -8 * r).all()
