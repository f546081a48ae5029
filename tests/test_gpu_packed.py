"""Packed sequences on the GPU (rope_packed, attn_fwd_packed, attn_bwd_packed) against the 64-bit
reference of tests/packed_ref.py: rotations bit for bit, attention and gradients within the bounds
derived there."""
import math

import pytest
import torch

import attention_pipelining_gb300 as ap
from tests import packed_ref as ref
from tests.test_packed_host import CUT_KEYS, CUT_TILES

pytestmark = pytest.mark.gpu

BAD_INDEX = 6
MARK = 7.0    # what outputs hold before a call


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


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(H_q, H_kv, D, lens_q, lens_k=None, lead=0, pad=0, seed=0, kscale=1.0, poison=True):
    """Views of one tensor; tokens of no sequence (``lead`` before the first, ``pad`` behind the
    last) hold infinities and NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cu_q = [lead + c for c in ref.bounds(lens_q)]
    cu_k = cu_q if lens_k is None else [lead + c for c in ref.bounds(lens_k)]
    T_q, T_k = max(1, cu_q[-1] + pad), max(1, cu_k[-1] + pad)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k, v, do = r(T_q, H_q, D), r(T_k, H_kv, D) * kscale, r(T_k, H_kv, D), r(T_q, H_q, D)
    for x, cu in ((q, cu_q), (k, cu_k), (v, cu_k), (do, cu_q)):
        if poison:
            for y in (x[:cu[0]], x[cu[-1]:]):
                y[:, :, 0::3], y[:, :, 1::3], y[:, :, 2::3] = math.inf, math.nan, -math.inf
    if lens_k is None:
        x = torch.cat([q, k, v], 1).bfloat16()
        q, k, v = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
    else:
        x = torch.cat([k, v], 1).bfloat16()
        q, k, v = q.bfloat16(), x[:, :H_kv], x[:, H_kv:]
    return q, k, v, do.bfloat16(), cu_q, cu_k


def filled(*shape, dtype=torch.bfloat16):
    return torch.full(shape, MARK, dtype=dtype, device="cuda")


def forward(q, k, v, cu_q, cu_k, causal, scale, **kw):
    out = (filled(*q.shape), filled(q.shape[1], q.shape[0], dtype=torch.float32))
    return ap.attn_fwd_packed(q, k, v, ints(cu_q), causal, scale, cu_k=None if cu_k is cu_q else ints(cu_k),
                              out=out, **kw)


def check_forward(q, k, v, cu_q, cu_k, causal, scale, got, what=""):
    o, lse = got
    ro, rl, to, tl = ref.forward(q.double(), k.double(), v.double(), cu_q, cu_k, causal, scale)
    inside = slice(cu_q[0], cu_q[-1])
    for x in (o[:cu_q[0]], o[cu_q[-1]:], lse[:, :cu_q[0]], lse[:, cu_q[-1]:]):
        assert (x == MARK).all(), (what, "rows of no sequence changed")
    o, ro, to = o[inside].double(), ro[inside], to[inside]
    off = (o - ro).abs()
    assert torch.isfinite(o).all(), what
    assert (off <= to).all(), (what, (off - to).argmax(), (off / to).max().item())
    lse, rl, tl = lse[:, inside].double(), rl[:, inside], tl[:, inside]
    none = torch.isinf(rl)
    assert torch.equal(lse[none], rl[none]), what
    off = (lse - rl).abs()[~none]
    assert (off <= tl[~none]).all(), (what, off.max().item(), tl[~none].min().item())


def backward(q, k, v, o, lse, do, cu_q, cu_k, causal, scale, **kw):
    out = (filled(*q.shape), filled(*k.shape), filled(*v.shape))
    return ap.attn_bwd_packed(q, k, v, o, lse, do, ints(cu_q), causal, scale,
                              cu_k=None if cu_k is cu_q else ints(cu_k), out=out, **kw)


def check_backward(q, k, v, o, lse, do, cu_q, cu_k, causal, scale, got, what=""):
    want = ref.backward(q.double(), k.double(), v.double(), o.double(), lse.double(), do.double(), cu_q, cu_k,
                        causal, scale)
    for (name, (r, allow, sd)), x, cu in zip(want.items(), got, (cu_q, cu_k, cu_k)):
        for y in (x[:cu[0]], x[cu[-1]:]):
            assert (y == MARK).all(), (what, name, "rows of no sequence changed")
        x, r, allow, sd = (t[cu[0]:cu[-1]].double() for t in (x, r, allow, sd))
        assert torch.isfinite(x).all(), (what, name)
        off = (x - r).abs()
        assert (off <= allow).all(), (what, name, (off / allow).max().item(), off.max().item())
        live = sd > 1e-30
        if live.any():   # the model bounds each rounding's deviation: no more than that on average
            z = (off[live] / sd[live]).square().mean().sqrt().item()
            assert z <= 1.5, (what, name, z)


CASES = [
    # H_q, H_kv, D, lens_q, lens_k, causal, scale, kscale
    (32, 8, 128, [100], None, True, 0.088, 1.0),
    (4, 4, 64, [1], None, True, 0.125, 1.0),
    (2, 2, 128, [128, 129, 127, 1, 0, 256, 257], None, True, 0.088, 1.0),
    (4, 2, 64, [63, 64, 65, 0, 0, 300], None, True, 0.125, 3.0),
    (8, 1, 128, [31, 33, 500], None, False, 0.088, 1.0),
    (10, 2, 128, [37, 0, 64, 300, 24, 48], None, True, 0.088, 1.0),
    (7, 1, 64, [1, 2, 3, 16, 17, 400], None, True, 0.125, 1.0),
    (3, 1, 128, [40, 41, 79, 81, 200], None, False, 0.088, 1.0),
    (12, 2, 64, [19, 150], None, True, 0.125, 1.0),
    (16, 1, 64, [300, 9], None, True, 0.125, 1.0),
    (64, 1, 128, [70, 3], None, True, 0.088, 1.0),
    (40, 1, 64, [50, 2], None, True, 0.125, 1.0),
    (128, 1, 64, [20, 1], None, True, 0.125, 1.0),
    (31, 1, 128, [30, 5], None, False, 0.088, 1.0),
    # keys of other lengths: behind a prefix, fewer than queries (rows that see nothing), none, queries none
    (8, 2, 128, [1, 7, 64, 0, 130], [300, 7, 1000, 50, 131], True, 0.088, 1.0),
    (8, 2, 64, [200, 5, 70, 0], [60, 0, 200, 0], True, 0.125, 1.0),
    (4, 4, 128, [300, 129], [10, 128], True, 0.088, 1.0),
    (4, 2, 64, [70, 5, 0, 130], [200, 0, 33, 400], False, 0.125, 1.0),
    # scales of any sign
    (4, 2, 128, [90, 140], None, True, -0.3, 1.0),
    (4, 2, 64, [90, 140], None, False, 0.0, 1.0),
    # many short sequences
    (4, 1, 128, [(7 * i) % 23 for i in range(200)], None, True, 0.088, 1.0),
    (2, 2, 64, [(5 * i) % 11 for i in range(1500)], None, False, 0.125, 1.0),
]
IDS = [f"{c[0]}_{c[1]}_{c[2]}_{'causal' if c[5] else 'full'}_{n}" for n, c in enumerate(CASES)]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    H_q, H_kv, D, lens_q, lens_k, causal, scale, kscale = case
    for lead, pad in ((0, 0), (3, 130)):
        x = make(H_q, H_kv, D, lens_q, lens_k, lead, pad, kscale=kscale)
        q, k, v, _, cu_q, cu_k = x
        got = forward(q, k, v, cu_q, cu_k, causal, scale)
        check_forward(q, k, v, cu_q, cu_k, causal, scale, got, (lead, pad))


@pytest.mark.parametrize("case", [c for c in CASES if len(c[3]) < 32],
                         ids=[i for i, c in zip(IDS, CASES) if len(c[3]) < 32])
def test_forward_among_many_tokens(case):
    """Few tokens take one kernel, more of them a plan before it: the same results to the bit, also for bounds
    that are not in order."""
    H_q, H_kv, D, lens_q, lens_k, causal, scale, kscale = case
    pad = 256 * 152   # (a tile holds 256 positions at most, a device has 152 multiprocessors)
    q, k, v, _, cu_q, cu_k = make(H_q, H_kv, D, lens_q, lens_k, kscale=kscale)
    more = [torch.cat([x, x.new_full((pad, *x.shape[1:]), math.nan)]) for x in (q, k, v)]
    few = forward(q, k, v, cu_q, cu_k, causal, scale)
    many = forward(*more, cu_q, cu_k, causal, scale)
    n = q.shape[0]
    assert torch.equal(many[0][:n], few[0]) and torch.equal(many[1][:, :n], few[1])
    if len(cu_q) > 2:
        swapped = cu_q[:-2] + [cu_q[-1], cu_q[-2]]
        ends = [0] + [cu_k[-1]] * (len(cu_k) - 1)
        few = forward(q, k, v, swapped, ends, causal, scale)
        many = forward(*more, swapped, ends, causal, scale)
        assert torch.equal(many[0][:n], few[0]) and torch.equal(many[1][:, :n], few[1])
        torch.cuda.synchronize()
        assert ap.device_status(reset=True) == (BAD_INDEX if cu_q[-1] > cu_q[-2] else 0)


@pytest.mark.parametrize("det", [False, True], ids=["atomic", "deterministic"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case, det):
    H_q, H_kv, D, lens_q, lens_k, causal, scale, kscale = case
    for lead, pad in ((0, 0), (3, 130)):
        q, k, v, do, cu_q, cu_k = make(H_q, H_kv, D, lens_q, lens_k, lead, pad, kscale=kscale)
        o, lse = forward(q, k, v, cu_q, cu_k, causal, scale)
        got = backward(q, k, v, o, lse, do, cu_q, cu_k, causal, scale, deterministic=det)
        check_backward(q, k, v, o, lse, do, cu_q, cu_k, causal, scale, got, (lead, pad))


@pytest.mark.parametrize("D,H_q,H_kv,causal", [(128, 8, 2, True), (64, 4, 4, False)])
def test_longer_sequences(D, H_q, H_kv, causal):
    lens = [2500, 1100, 3]
    q, k, v, do, cu, _ = make(H_q, H_kv, D, lens, pad=5)
    o, lse = forward(q, k, v, cu, cu, causal, D ** -0.5)
    check_forward(q, k, v, cu, cu, causal, D ** -0.5, (o, lse))
    for det in (False, True):
        got = backward(q, k, v, o, lse, do, cu, cu, causal, D ** -0.5, deterministic=det)
        check_backward(q, k, v, o, lse, do, cu, cu, causal, D ** -0.5, got)


@pytest.mark.parametrize("D", [64, 128])
def test_as_attn_fwd_and_attn_bwd(D):
    """Sequences of one length against the calls that take [B, H, S, D]: twice the rounding model apart
    at most, LSE to fp32."""
    B, S, H_q, H_kv = 3, 700, 8, 2
    q, k, v, do, cu, _ = make(H_q, H_kv, D, [S] * B)
    scale = D ** -0.5
    o, lse = forward(q, k, v, cu, cu, True, scale)
    got = backward(q, k, v, o, lse, do, cu, cu, True, scale)
    b = [t.reshape(B, S, -1, D).transpose(1, 2).contiguous() for t in (q, k, v, o, do)]
    o2, lse2 = ap.attn_fwd(*b[:3], True, scale)
    assert (lse.view(H_q, B, S).transpose(0, 1) - lse2).abs().max() <= 2.0 ** -19 * (1 + lse2.abs().max())
    _, _, tol, _ = ref.forward(q.double(), k.double(), v.double(), cu, cu, True, scale)
    assert ((b[3] - o2).transpose(1, 2).reshape(B * S, H_q, D).abs() <= 2 * tol).all()
    want = ref.backward(q.double(), k.double(), v.double(), o.double(), lse.double(), do.double(), cu, cu, True, scale)
    g2 = ap.attn_bwd(*b[:4], lse.view(H_q, B, S).transpose(0, 1).contiguous(), b[4], True, scale)
    for (name, (_, allow, _)), x, y in zip(want.items(), got, g2):
        assert ((x.double() - y.transpose(1, 2).reshape(x.shape).double()).abs() <= 2 * allow).all(), name


# ---------------------------------------------------------------- what sequences do not see of one another


@pytest.mark.parametrize("D,H_q,H_kv", [(128, 8, 2), (64, 5, 1), (64, 4, 4)])
@pytest.mark.parametrize("causal", [True, False])
def test_a_sequence_s_infinities_stay_its_own(D, H_q, H_kv, causal):
    """Every second sequence of NaN and infinities: the others' results are those without them, bit
    for bit (dq by the deterministic path; by atomics within the bounds)."""
    lens = [70, 130, 1, 200, 128, 64, 3, 90]
    q, k, v, do, cu, _ = make(H_q, H_kv, D, lens)
    scale = D ** -0.5
    o, lse = forward(q, k, v, cu, cu, causal, scale)
    clean = backward(q, k, v, o, lse, do, cu, cu, causal, scale, deterministic=True)
    bad = [t.clone() for t in (q, k, v, do, o)]
    bad_lse = lse.clone()
    good = torch.ones(cu[-1], dtype=torch.bool, device="cuda")
    for b in range(1, len(lens), 2):
        rows = slice(cu[b], cu[b + 1])
        good[rows] = False
        for t in bad:
            t[rows, :, 0::3], t[rows, :, 1::3], t[rows, :, 2::3] = math.inf, math.nan, -math.inf
        bad_lse[:, rows] = math.nan
    o2, lse2 = forward(*bad[:3], cu, cu, causal, scale)
    assert torch.equal(o2[good], o[good]) and torch.equal(lse2[:, good], lse[:, good])
    assert not torch.isfinite(o2[~good]).any()
    got = backward(*bad[:3], bad[4], bad_lse, bad[3], cu, cu, causal, scale, deterministic=True)
    for x, y in zip(got, clean):
        assert torch.equal(x[good], y[good])
    got = backward(*bad[:3], bad[4], bad_lse, bad[3], cu, cu, causal, scale)
    assert torch.equal(got[1][good], clean[1][good]) and torch.equal(got[2][good], clean[2][good])
    want = ref.backward(q.double(), k.double(), v.double(), o.double(), lse.double(), do.double(), cu, cu, causal, scale)
    r, allow, _ = want["dq"]
    assert ((got[0].double() - r).abs() <= allow)[good].all()


def test_bounds_that_are_not_in_order():
    """Entries below 0, below the one before or above T are taken as the nearest in order, and recorded."""
    q, k, v, do, _, _ = make(4, 2, 64, [400])
    for cu, taken in (([-5, 100, 400], [0, 100, 400]), ([0, 300, 200, 400], [0, 300, 300, 400]),
                      ([10, 2 ** 31 - 1, 50], [10, 400, 400]), ([-2 ** 31, -7, -1], [0, 0, 0]),
                      ([0, 400] * 40, [0] + [400] * 79), ([401, 500], [400, 400])):
        o, lse = forward(q, k, v, cu, cu, True, 0.125)
        torch.cuda.synchronize()
        assert ap.device_status(reset=True) == BAD_INDEX
        check_forward(q, k, v, taken, taken, True, 0.125, (o, lse), cu)
        for det in (False, True):
            got = backward(q, k, v, o, lse, do, cu, cu, True, 0.125, deterministic=det)
            torch.cuda.synchronize()
            assert ap.device_status(reset=True) == BAD_INDEX
            check_backward(q, k, v, o, lse, do, taken, taken, True, 0.125, got, cu)
    q, k, v, do, _, _ = make(4, 2, 64, [100], [300])
    o, lse = forward(q, k, v, [0, 100], [0, 301], True, 0.125)
    torch.cuda.synchronize()
    assert ap.device_status(reset=True) == BAD_INDEX
    check_forward(q, k, v, [0, 100], [0, 300], True, 0.125, (o, lse))


# ---------------------------------------------------------------- how it is called


def views(H, D, T, order):
    """A [T, H, D] view whose dimensions lie in another order, or apart."""
    if order == "heads first":
        return torch.empty(H, T, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    if order == "apart":
        return torch.empty(T + 2, H + 3, D + 8, dtype=torch.bfloat16, device="cuda")[1:-1, 1:-2, :D]
    return torch.empty(T, 2 * H, D, dtype=torch.bfloat16, device="cuda")[:, ::2]


@pytest.mark.parametrize("order", ["heads first", "apart", "every second head"])
def test_strides(order):
    D, H_q, H_kv, lens = 128, 6, 2, [50, 200, 3]
    q, k, v, do, cu, _ = make(H_q, H_kv, D, lens, pad=4, poison=False)
    o, lse = forward(q, k, v, cu, cu, True, 0.088)
    g = backward(q, k, v, o, lse, do, cu, cu, True, 0.088, deterministic=True)
    q2, k2, v2, do2, o2, dq, dk, dv = (
        views(t.shape[1], D, t.shape[0], order).copy_(t) for t in (q, k, v, do, o, q, k, v))
    o2.fill_(MARK)
    ap.attn_fwd_packed(q2, k2, v2, ints(cu), True, 0.088, out=(o2, lse.clone()))
    assert torch.equal(o2, o)
    for x in (dq, dk, dv):
        x.fill_(MARK)
    ap.attn_bwd_packed(q2, k2, v2, o2, lse, do2, ints(cu), True, 0.088, out=(dq, dk, dv), deterministic=True)
    for x, y in zip((dq, dk, dv), g):
        assert torch.equal(x, y)


def test_gradients_into_one_buffer():
    """dq, dk and dv as views of the projection's gradient [T, (H_q + 2 H_kv) D]."""
    H_q, H_kv, D = 8, 2, 64
    q, k, v, do, cu, _ = make(H_q, H_kv, D, [77, 200], pad=2)
    o, lse = forward(q, k, v, cu, cu, True, 0.125)
    g = backward(q, k, v, o, lse, do, cu, cu, True, 0.125, deterministic=True)
    x = filled(q.shape[0], H_q + 2 * H_kv, D)
    out = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
    ap.attn_bwd_packed(q, k, v, o, lse, do, ints(cu), True, 0.125, out=out, deterministic=True)
    assert torch.equal(x, torch.cat(g, 1))


def test_allocated_outputs_hold_zeros_elsewhere():
    q, k, v, do, cu, _ = make(4, 2, 64, [30, 50], lead=2, pad=9)
    o, lse = ap.attn_fwd_packed(q, k, v, ints(cu), True, 0.125)
    ws = torch.empty(ap.packed_workspace_bytes(2, *[q.shape[0]] * 2, 4, 2, 64), dtype=torch.uint8, device="cuda")
    o2, lse2 = forward(q, k, v, cu, cu, True, 0.125, workspace=ws)
    inside = slice(cu[0], cu[-1])
    assert torch.equal(o[inside], o2[inside]) and torch.equal(lse[:, inside], lse2[:, inside])
    assert o[:2].eq(0).all() and o[-9:].eq(0).all() and lse[:, :2].eq(0).all() and lse[:, -9:].eq(0).all()
    for det in (False, True):
        n = ap.packed_bwd_workspace_bytes(2, *[q.shape[0]] * 2, 4, 2, 64, det)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")     # NaN throughout
        got = ap.attn_bwd_packed(q, k, v, o, lse, do, ints(cu), True, 0.125, deterministic=det, workspace=ws)
        for x in got:
            assert x[:2].eq(0).all() and x[-9:].eq(0).all()
        want = ref.backward(*(t.double() for t in (q, k, v, o, lse, do)), cu, cu, True, 0.125)
        for (name, (r, allow, _)), x in zip(want.items(), got):
            assert ((x.double() - r).abs() <= allow)[inside].all(), (name, det)


@pytest.mark.parametrize("D", [64, 128])
def test_results_are_the_same_each_time(D):
    q, k, v, do, cu, _ = make(8, 2, D, [(37 * i) % 300 for i in range(40)])
    first = None
    for n in range(4):
        o, lse = forward(q, k, v, cu, cu, True, 0.1)
        got = (o, lse, *backward(q, k, v, o, lse, do, cu, cu, True, 0.1, deterministic=True),
               *backward(q, k, v, o, lse, do, cu, cu, True, 0.1)[1:])
        first = first or [t.clone() for t in got]
        for x, y in zip(first, got):
            assert torch.equal(x, y), n


def test_a_captured_step_follows_its_bounds():
    """Rotation, attention and gradients in a graph; the bounds change between replays, and two graphs
    with workspaces of their own run at once."""
    H_q, H_kv, D, T, B = 8, 2, 128, 600, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H_q + 2 * H_kv, D, generator=g, device="cuda").bfloat16()
    q, k, v = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
    do = torch.randn(T, H_q, D, generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 64, (3, T), generator=g, device="cuda", dtype=torch.int32)
    ang = torch.arange(64, device="cuda")[:, None] * 0.7 ** torch.arange(64, device="cuda")
    cos, sin, sec = torch.cos(ang), torch.sin(ang), (16, 24, 24)

    def step(cu):
        a, b = ap.rope_packed(q, k, pos, cos, sin, sec)
        o, lse = ap.attn_fwd_packed(a, b, v, cu, True, 0.088)
        dq, dk, dv = ap.attn_bwd_packed(a, b, v, o, lse, do, cu, True, 0.088, deterministic=True)
        dq, dk = ap.rope_packed(dq, dk, pos, cos, sin, sec, inverse=True, out=(dq, dk))
        return o, lse, dq, dk, dv

    graphs = []
    for n in range(2):
        cu, s = ints([0] * (B + 1)), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step(cu)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = step(cu)
        graphs.append((graph, cu, s, out))
    lists = [[0, 100, 100, 250, 600], [0, 1, 2, 3, 4], [0, 600, 600, 600, 600], [5, 155, 300, 301, 590]]
    for n in range(4):
        picks = lists[n], lists[(n + 1) % 4]
        for (graph, cu, s, _), c in zip(graphs, picks):
            cu.copy_(ints(c))
        torch.cuda.synchronize()
        for graph, _, s, _ in graphs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (_, cu, _, out), c in zip(graphs, picks):
            for a, b in zip(out, step(ints(c))):
                assert torch.equal(a, b), c


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("n", [3, 40])
def test_calls_after_one_another_in_one_workspace(n, deterministic):
    """Calls queued without a pause, each with bounds that the copy before it brings, in one workspace."""
    lens = [[(37 * i + 90 * j) % 211 for i in range(n)] for j in range(2)]
    total = max(sum(x) for x in lens)
    sets = []
    for x in lens:
        x[-1] += total - sum(x)
        sets.append(ints(ref.bounds(x)))
    q, k, v, do, _, _ = make(8, 2, 64, [total])
    sizes = (n, total, total, 8, 2, 64)
    fw = torch.empty(ap.packed_workspace_bytes(*sizes), dtype=torch.uint8, device="cuda")
    bw = torch.empty(ap.packed_bwd_workspace_bytes(*sizes, deterministic), dtype=torch.uint8, device="cuda")

    def step(cu):
        o, lse = ap.attn_fwd_packed(q, k, v, cu, True, 0.125, workspace=fw)
        return o, lse, *ap.attn_bwd_packed(q, k, v, o, lse, do, cu, True, 0.125, workspace=bw,
                                           deterministic=deterministic)

    want = []
    for cu in sets:
        want.append(step(cu))
        torch.cuda.synchronize()
    cu, got = sets[0].clone(), []
    for i in range(24):
        cu.copy_(sets[i % 2])
        got.append(step(cu))
    for i, x in enumerate(got):
        for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), x, want[i % 2]):
            # dq's fp32 sums may come in another order: one step of bf16 (2^-7 of the value at most)
            # where that crosses a tie, and what the sums themselves differ by near zero
            if name == "dq" and not deterministic:
                scale = b.float().abs().max()
                assert ((a.float() - b.float()).abs() <= b.float().abs() * 2.0 ** -7 + scale * 2.0 ** -18).all(), i
            else:
                assert torch.equal(a, b), (i, name)


def test_streams_and_two_calls_at_once():
    q, k, v, do, cu, _ = make(8, 2, 128, [400, 700, 100])
    want = forward(q, k, v, cu, cu, True, 0.088)
    grads = backward(q, k, v, *want, do, cu, cu, True, 0.088, deterministic=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    cu_d, got = ints(cu), []
    torch.cuda.synchronize()
    for n in range(9):
        s = streams[n % 3]
        o, lse = ap.attn_fwd_packed(q, k, v, cu_d, True, 0.088, stream=s)
        got.append((o, lse, *ap.attn_bwd_packed(q, k, v, o, lse, do, cu_d, True, 0.088, deterministic=True,
                                                stream=s)))
    torch.cuda.synchronize()
    for x in got:
        for a, b in zip(x, (*want, *grads)):
            assert torch.equal(a, b)


def test_tokens_beyond_32_bit_offsets():
    """A sequence behind 2^31 elements of q, o and the gradients, and behind 2^32 bytes."""
    H_q, H_kv, D, T = 16, 2, 128, (1 << 20) + 777
    n = 333
    q = torch.zeros(T, H_q, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(T, H_kv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q1, k1, v1, do1, cu1, _ = make(H_q, H_kv, D, [n], seed=5)
    do, at = torch.zeros_like(q), T - n
    for x, y in ((q, q1), (k, k1), (v, v1), (do, do1)):
        x[at:] = y
    cu = [at, T]
    o, lse = ap.attn_fwd_packed(q, k, v, ints(cu), True, 0.088)
    o1, lse1 = forward(q1, k1, v1, cu1, cu1, True, 0.088)
    assert torch.equal(o[at:], o1) and torch.equal(lse[:, at:], lse1)
    want = backward(q1, k1, v1, o1, lse1, do1, cu1, cu1, True, 0.088, deterministic=True)
    for det in (True, False):
        got = ap.attn_bwd_packed(q, k, v, o, lse, do, ints(cu), True, 0.088, deterministic=det)
        for i, (x, y) in enumerate(zip(got, want)):
            if i == 0 and not det:
                r, allow, _ = ref.backward(*(t.double() for t in (q1, k1, v1, o1, lse1, do1)), cu1, cu1, True,
                                           0.088)["dq"]
                assert ((x[at:].double() - r).abs() <= allow).all()
            else:
                assert torch.equal(x[at:], y)
        del got
    pos = torch.zeros(1, T, dtype=torch.int32, device="cuda")
    pos[0, at:] = torch.arange(n, dtype=torch.int32, device="cuda")
    ang = torch.arange(n, device="cuda")[:, None] * 0.9 ** torch.arange(64, device="cuda")
    a, b = ap.rope_packed(q, k, pos, torch.cos(ang), torch.sin(ang), out=(o, k))
    c, d = ap.rope_packed(q1, k1, pos[:, at:].contiguous(), torch.cos(ang), torch.sin(ang))
    assert torch.equal(a[at:], c) and torch.equal(b[at:], d)


CUT = [
    # H_q, H_kv, D, lens_q, lens_k, causal: tiles of long sequences, and the key blocks that few
    # tiles see, are cut into parts where there are few (from CUT_KEYS blocks of keys, and CUT_TILES
    # query tiles, on)
    (8, 2, 128, [3, 1], [5000, 40], True),
    (4, 4, 64, [1, 130, 0], [9000, 2100, 3000], True),
    (8, 1, 128, [1500], None, True),
    (5, 1, 64, [700, 20], None, True),
    (2, 1, 128, [260], [1700], False),
    (4, 2, 64, [1100, 1], [1300, 700], False),
    (16, 1, 64, [40], [8200], True),
    (1, 1, 128, [2], [70000], False),      # as many parts as there may be
    (1, 1, 64, [70000], [2], False),
]


@pytest.mark.parametrize("case", CUT, ids=[f"{c[0]}_{c[1]}_{c[2]}_{c[3][0]}" for c in CUT])
def test_work_cut_into_parts(case):
    """Against the reference, and bit for bit the same each time, whichever part comes last."""
    H_q, H_kv, D, lens_q, lens_k, causal = case
    q, k, v, do, cu_q, cu_k = make(H_q, H_kv, D, lens_q, lens_k, lead=1, pad=70, seed=11)
    scale = D ** -0.5
    o, lse = forward(q, k, v, cu_q, cu_k, causal, scale)
    check_forward(q, k, v, cu_q, cu_k, causal, scale, (o, lse))
    first = None
    for det in (True, False, True):
        got = backward(q, k, v, o, lse, do, cu_q, cu_k, causal, scale, deterministic=det)
        check_backward(q, k, v, o, lse, do, cu_q, cu_k, causal, scale, got, det)
        first = first or [t.clone() for t in got]
        for x, y in zip(first if det else first[1:], got if det else got[1:]):
            assert torch.equal(x, y)
    for _ in range(3):
        for x, y in zip(forward(q, k, v, cu_q, cu_k, causal, scale), (o, lse)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("off", [-1, 0, 1])
def test_around_the_least_parts(D, off):
    """Works of one block less than is cut, of as many, and of one more; the last block of one key or
    query, or full."""
    scale = D ** -0.5
    for last in (1, 128):
        m, n = ((blocks + off - 1) * 128 + last for blocks in (CUT_KEYS, CUT_TILES[D]))
        for lens_q, lens_k, causal in (([5, 0, 2], [m, 30, 9], True), ([n], [40], False), ([n, 3], [n, 3], True)):
            q, k, v, do, cu_q, cu_k = make(2, 1, D, lens_q, lens_k, pad=1, seed=m)
            if lens_q[0] == n:   # (a tile of one head's 128 tokens)
                q, do = q[:, :1], do[:, :1]
            o, lse = forward(q, k, v, cu_q, cu_k, causal, scale)
            check_forward(q, k, v, cu_q, cu_k, causal, scale, (o, lse))
            first = None
            for det in (True, False, True):
                got = backward(q, k, v, o, lse, do, cu_q, cu_k, causal, scale, deterministic=det)
                check_backward(q, k, v, o, lse, do, cu_q, cu_k, causal, scale, got, det)
                first = first or [t.clone() for t in got]
                for x, y in zip(first if det else first[1:], got if det else got[1:]):
                    assert torch.equal(x, y)


@pytest.mark.parametrize("B", [31, 32, 1023, 1024, 2047, 2048, 5000])
def test_any_number_of_sequences(B):
    """Around the numbers at which the plan changes its way of going through them."""
    lens_q = [(3 * i) % 5 for i in range(B)]
    lens_k = [(7 * i) % 4 + (i % 97 == 0) * 50 for i in range(B)]
    for lk in (None, lens_k):
        q, k, v, do, cu_q, cu_k = make(1, 1, 64, lens_q, lk, pad=3)
        o, lse = forward(q, k, v, cu_q, cu_k, False, 0.125)
        check_forward(q, k, v, cu_q, cu_k, False, 0.125, (o, lse))
        got = backward(q, k, v, o, lse, do, cu_q, cu_k, False, 0.125)
        check_backward(q, k, v, o, lse, do, cu_q, cu_k, False, 0.125, got)


# heads a key head: above 32 with spare rows (one or more tokens a tile), without, and just 32
LARGE = [(32, 1, [1, 2, 7, 8, 9, 33]), (64, 2, [4, 17]), (36, 1, [5, 6, 7, 50]), (96, 1, [1, 2, 3, 40, 41]),
         (192, 2, [2, 33]), (100, 1, [1, 2, 31]), (124, 1, [2, 3, 20])]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H_q,H_kv,lens", LARGE, ids=[f"{c[0]}_{c[1]}" for c in LARGE])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_large_groups(H_q, H_kv, lens, D, causal):
    """Tiles of one to four tokens, odd and even numbers of them: against the reference, and the same bits
    again and again, also behind many tokens (where a plan comes first)."""
    q, k, v, do, cu, _ = make(H_q, H_kv, D, lens, lead=1, pad=3, seed=H_q)
    scale = D ** -0.5
    o, lse = forward(q, k, v, cu, cu, causal, scale)
    check_forward(q, k, v, cu, cu, causal, scale, (o, lse))
    for _ in range(20):
        a, b = forward(q, k, v, cu, cu, causal, scale)
        assert torch.equal(a, o) and torch.equal(b, lse)
    pad = 304 * (128 * H_kv // H_q)   # (more tiles than a device has multiprocessors)
    more = [torch.cat([x, x.new_full((pad, *x.shape[1:]), math.nan)]) for x in (q, k, v)]
    a, b = forward(*more, cu, cu, causal, scale)
    assert torch.equal(a[:-pad], o) and torch.equal(b[:, :-pad], lse)
    for det in (False, True):
        got = backward(q, k, v, o, lse, do, cu, cu, causal, scale, deterministic=det)
        check_backward(q, k, v, o, lse, do, cu, cu, causal, scale, got, det)


def test_more_tiles_than_thread_blocks_keep():
    """The forward's thread blocks keep 64 tiles each: with more, there are more of them.  The same
    heads in two calls are the reference."""
    H, D, lens = 128, 64, [5 + i % 3 for i in range(100)]
    q, k, v, do, cu, _ = make(H, H, D, lens)
    o, lse = forward(q, k, v, cu, cu, True, 0.125)
    g = backward(q, k, v, o, lse, do, cu, cu, True, 0.125)
    for h in (slice(0, 64), slice(64, 128)):
        a = forward(q[:, h], k[:, h], v[:, h], cu, cu, True, 0.125)
        assert torch.equal(o[:, h], a[0]) and torch.equal(lse[h], a[1])
        b = backward(q[:, h], k[:, h], v[:, h], o[:, h], lse[h].contiguous(), do[:, h], cu, cu, True, 0.125)
        for x, y in zip(g[1:], b[1:]):
            assert torch.equal(x[:, h], y)


def test_tensors_that_only_the_call_holds():
    """Bounds and positions made in the call's own argument list live as long as the call needs them,
    whatever memory it allocates itself."""
    q, k, v, do, cu, _ = make(2, 1, 64, [(5 * i) % 9 for i in range(600)])
    o, lse = forward(q, k, v, cu, cu, True, 0.125)
    for _ in range(20):
        a, b = ap.attn_fwd_packed(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), True, 0.125,
                                  cu_k=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert torch.equal(a, o) and torch.equal(b, lse)


@pytest.mark.parametrize("D,H_q,H_kv", [(128, 4, 1), (64, 2, 2)])
@pytest.mark.parametrize("what", ["forward", "backward", "deterministic"])
def test_a_wait_that_runs_out(D, H_q, H_kv, what):
    """A signal withheld: every role unwinds, the status word says so, and the next call works."""
    from attention_pipelining_gb300 import packed
    q, k, v, do, cu, _ = make(H_q, H_kv, D, [300, 700, 40])
    o, lse = forward(q, k, v, cu, cu, True, 0.1)
    c = ints(cu)
    if what == "forward":
        packed.fwd_packed_timeout_test(q, k, v, c, True, 0.1, drop_block=1)
    else:
        packed.bwd_packed_timeout_test(q, k, v, o, lse, do, c, True, 0.1, drop_item=1,
                                       deterministic=what == "deterministic")
    torch.cuda.synchronize()
    assert ap.device_status(reset=True) == 5
    a = forward(q, k, v, cu, cu, True, 0.1)
    assert torch.equal(a[0], o) and torch.equal(a[1], lse)
    got = backward(q, k, v, o, lse, do, cu, cu, True, 0.1)
    check_backward(q, k, v, o, lse, do, cu, cu, True, 0.1, got)


@pytest.mark.parametrize("D", [64, 128])
def test_a_wait_that_runs_out_in_cut_work(D):
    """The same where a plan cuts tiles into parts: what they counted does not reach the next call in
    the same workspace."""
    from attention_pipelining_gb300 import packed
    q, k, v, do, cu, _ = make(4, 2, D, [2500, 700])
    ws = torch.full((max(ap.packed_workspace_bytes(2, 3200, 3200, 4, 2, D),
                         ap.packed_bwd_workspace_bytes(2, 3200, 3200, 4, 2, D, True)),), 255,
                    dtype=torch.uint8, device="cuda")
    o, lse = forward(q, k, v, cu, cu, True, 0.1, workspace=ws)
    check_forward(q, k, v, cu, cu, True, 0.1, (o, lse))
    want = backward(q, k, v, o, lse, do, cu, cu, True, 0.1, workspace=ws, deterministic=True)
    for _ in range(2):
        packed.fwd_packed_timeout_test(q, k, v, ints(cu), True, 0.1, drop_block=5, workspace=ws)
        torch.cuda.synchronize()
        assert ap.device_status(reset=True) == 5
        a = forward(q, k, v, cu, cu, True, 0.1, workspace=ws)
        assert torch.equal(a[0], o) and torch.equal(a[1], lse)
        packed.bwd_packed_timeout_test(q, k, v, o, lse, do, ints(cu), True, 0.1, drop_item=1, workspace=ws,
                                       deterministic=True)
        torch.cuda.synchronize()
        assert ap.device_status(reset=True) == 5
        got = backward(q, k, v, o, lse, do, cu, cu, True, 0.1, workspace=ws, deterministic=True)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


# ---------------------------------------------------------------- rotation

ROPE = [
    # T, H_q, H_kv, D, sections, rot, interleaved
    (1, 4, 1, 128, (64,), 128, False),
    (32, 32, 8, 128, (16, 24, 24), 128, False),
    (33, 5, 5, 64, (8, 12, 12), 64, False),
    (257, 3, 1, 64, (1, 2, 13), 32, True),
    (100, 2, 7, 128, (5, 11, 15, 33), 128, True),
    (9, 8, 8, 128, (3, 5), 16, False),
    (1000, 1, 1, 64, (31, 1), 64, False),
    (5000, 8, 2, 128, (30, 30, 4), 128, False),
]


def tables(rows, pairs, seed=2):
    inv = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return torch.cos(ang).float().cuda(), torch.sin(ang).float().cuda()


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", ROPE, ids=[str(c) for c in ROPE])
def test_rotation(case, inverse):
    """Bit for bit; out of place, in place, and into views; either of q and k alone."""
    T, H_q, H_kv, D, sections, rot, inter = case
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H_q + 2 * H_kv, D, generator=g, device="cuda").bfloat16()
    q, k = x[:, :H_q], x[:, H_q:H_q + H_kv]
    pos = torch.randint(0, 700, (len(sections), T), generator=g, device="cuda", dtype=torch.int32)
    cos, sin = tables(700, rot // 2)
    kw = dict(sections=sections, interleaved=inter, inverse=inverse)
    want = [ref.rope(t.double(), pos, cos, sin, sections, inter, inverse).bfloat16() for t in (q, k)]
    for a, b in zip(ap.rope_packed(q, k, pos, cos, sin, **kw), want):
        assert torch.equal(a, b)
    a, none = ap.rope_packed(q, None, pos, cos, sin, **kw)
    none2, b = ap.rope_packed(None, k, pos, cos, sin, **kw)
    assert none is None and none2 is None and torch.equal(a, want[0]) and torch.equal(b, want[1])
    was = x.clone()
    ap.rope_packed(q, k, pos, cos, sin, out=(q, k), **kw)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(x[:, H_q + H_kv:], was[:, H_q + H_kv:])


def test_rotation_s_positions_out_of_range():
    """A token with a position outside the tables keeps its output rows; the others do not mind."""
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(40, 3, 64, generator=g, device="cuda").bfloat16()
    k = torch.randn(40, 2, 64, generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 50, (2, 40), generator=g, device="cuda", dtype=torch.int32)
    cos, sin = tables(50, 32)
    for axis, t, x in ((0, 3, -1), (1, 17, 50), (0, 39, 2 ** 31 - 1), (1, 0, -2 ** 31)):
        pos[axis, t] = x
    out = filled(40, 3, 64), filled(40, 2, 64)
    ap.rope_packed(q, k, pos, cos, sin, (20, 12), out=out)
    torch.cuda.synchronize()
    assert ap.device_status(reset=True) == BAD_INDEX
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[3, 17, 39, 0]] = True
    for x, y in zip((q, k), out):
        want = ref.rope(x.double(), pos.clamp(0, 49), cos, sin, (20, 12), False, False).bfloat16()
        assert torch.equal(y[~bad], want[~bad]) and (y[bad] == MARK).all()


def test_rotation_of_values_that_are_not_finite():
    """They stay in their pair."""
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(8, 2, 64, generator=g, device="cuda").bfloat16()
    pos = torch.full((1, 8), 3, dtype=torch.int32, device="cuda")
    cos, sin = tables(50, 32)
    clean, _ = ap.rope_packed(q, None, pos, cos, sin)
    bad = q.clone()
    bad[2, 1, 5], bad[6, 0, 40] = math.nan, math.inf
    got, _ = ap.rope_packed(bad, None, pos, cos, sin)
    same = torch.ones_like(q, dtype=torch.bool)
    same[2, 1, [5, 37]] = False
    same[6, 0, [8, 40]] = False
    assert torch.equal(got[same], clean[same]) and not torch.isfinite(got[~same]).any()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_of_tiny_values(interleaved):
    """Where the products' last bits lie below fp32's smallest step, 2^-149: each product's error, and
    each sum's, is rounded to that, by 2^-150 at most; four of them, beside the one rounding to
    bf16 (2^-8 of the value, or half of its smallest step, 2^-134)."""
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn(400, 2, 64, generator=g, device="cuda") * 2.0 ** torch.randint(
        -134, -100, (400, 1, 64), generator=g, device="cuda")
    q = q.bfloat16()
    assert (q.abs() < 2.0 ** -126).any() and (q != 0).any()
    pos = torch.randint(0, 50, (1, 400), generator=g, device="cuda", dtype=torch.int32)
    cos, sin = tables(50, 32)
    got, _ = ap.rope_packed(q, None, pos, cos, sin, interleaved=interleaved)
    x, c, s = q.double(), cos.double()[pos[0].long()][:, None], sin.double()[pos[0].long()][:, None]
    u, w = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    first, second = u * c - w * s, w * c + u * s     # (doubles are exact to 2^-53 of the products)
    want = torch.stack([first, second], -1).flatten(2) if interleaved else torch.cat([first, second], -1)
    off = (got.double() - want).abs()
    assert (off <= torch.maximum(want.abs() * 2.0 ** -8, torch.full_like(want, 2.0 ** -134)) + 2.0 ** -148).all()


def test_rotation_s_gradient_against_differences():
    """sum(w rope(x)) changes by the inverse rotation of w (whole numbers, so that only the two
    roundings differ)."""
    g = torch.Generator(device="cuda").manual_seed(6)
    w = torch.randn(20, 4, 128, generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 90, (3, 20), generator=g, device="cuda", dtype=torch.int32)
    cos, sin = tables(90, 64)
    sec = (10, 20, 34)
    grad, _ = ap.rope_packed(w, None, pos, cos, sin, sec, inverse=True)
    for d in range(0, 128, 7):
        x = torch.zeros_like(w)
        x[..., d] = 1.0
        y, _ = ap.rope_packed(x, None, pos, cos, sin, sec)
        diff = (w.double() * y.double()).sum(-1)
        # each of the two products' factors and the gradient are off by 2^-8 of themselves at most
        r = (w.double()[..., d % 64] ** 2 + w.double()[..., d % 64 + 64] ** 2).sqrt()
        assert ((diff - grad[..., d].double()).abs() <= 3 * 2.0 ** -8 * r).all()


# ---------------------------------------------------------------- together


def test_gradients_of_a_whole_step_against_differences():
    """Rotation, attention, back: the gradient of sum(w o) by the whole chain against the 64-bit
    chain's, within what the roundings of the rotated q and k, of o and of the gradients allow."""
    H_q, H_kv, D, lens = 4, 2, 64, [90, 33]
    q, k, v, w, cu, _ = make(H_q, H_kv, D, lens, seed=9)
    T = cu[-1]
    pos = torch.stack([torch.arange(T) // 9, torch.arange(T) % 9, torch.arange(T) % 4]).int().cuda()
    cos, sin = tables(64, 32)
    sec = (8, 12, 12)
    a, b = ap.rope_packed(q, k, pos, cos, sin, sec)
    o, lse = ap.attn_fwd_packed(a, b, v, ints(cu), True, 0.125)
    dq, dk, dv = ap.attn_bwd_packed(a, b, v, o, lse, w, ints(cu), True, 0.125)
    dq, dk = ap.rope_packed(dq, dk, pos, cos, sin, sec, inverse=True)

    def chain(x, y, z):
        def turn(t):
            axis = torch.tensor([0] * 8 + [1] * 12 + [2] * 12).cuda()
            at = pos.long()[axis].T
            c, s = (torch.gather(m.double(), 0, at)[:, None] for m in (cos, sin))
            u, r = t[..., :32], t[..., 32:]
            return torch.cat([u * c - r * s, r * c + u * s], -1)
        total = 0.0
        for n0, n1 in zip(cu, cu[1:]):
            for h in range(H_q):
                s = 0.125 * turn(x)[n0:n1, h] @ turn(y)[n0:n1, h // 2].T
                s = s.masked_fill(~ref.seen(n1 - n0, n1 - n0, True, "cuda"), -math.inf)
                total = total + (torch.softmax(s, 1) @ z[n0:n1, h // 2] * w[n0:n1, h].double()).sum()
        return total

    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    want = torch.autograd.grad(chain(*leaves), leaves)
    for name, x, y in zip(("dq", "dk", "dv"), (dq, dk, dv), want):
        # independent relative roundings of 2^-8 / sqrt(3) each: rotated q and k (each enters every score,
        # of size |s| <= 0.125 |q| |k| ~ 8), probabilities, dS, O, and the gradients twice.  Over the whole
        # tensor their root sum square is below 2^-8 (2 * 8 + 5) / sqrt(3) < 2^-4 of the gradient's norm.
        assert (x.double() - y).norm() <= 2.0 ** -4 * y.norm(), name
    # and a difference of the 64-bit chain along the computed gradient has that gradient's slope
    with torch.no_grad():
        d = dq.double() / dq.double().norm()
        slope = (chain(q.double() + 1e-4 * d, k.double(), v.double())
                 - chain(q.double() - 1e-4 * d, k.double(), v.double())) / 2e-4
        assert abs(slope - (d * want[0]).sum()) <= 1e-5 * abs(slope)


def test_refusals_on_the_device():
    q, k, v, do, cu, _ = make(4, 2, 64, [30, 50])
    c, lse = ints(cu), filled(4, 80, dtype=torch.float32)
    f = lambda **kw: ap.attn_fwd_packed(**{**dict(q=q, k=k, v=v, cu_q=c, causal=True, scale=0.1), **kw})  # noqa: E731
    for kw, e in ((dict(q=q.float()), TypeError), (dict(q=q[0]), TypeError), (dict(k=k.cpu()), TypeError),
                  (dict(k=k[:50]), ValueError), (dict(v=v[:50]), ValueError), (dict(v=v[:, :1]), ValueError),
                  (dict(cu_q=c.long()), TypeError), (dict(cu_q=c[:1]), TypeError), (dict(cu_q=c.cpu()), TypeError),
                  (dict(cu_k=c[:2]), TypeError), (dict(cu_q=ints([0, 1, 2, 3])[::2]), TypeError),
                  (dict(q=q.transpose(0, 2).contiguous().transpose(0, 2)), ValueError),
                  (dict(out=(q.contiguous(), lse[:, 1:])), TypeError), (dict(out=(q[:9], lse)), ValueError),
                  (dict(workspace=torch.empty(9, device="cuda")), TypeError), (dict(scale=math.nan), ap.AttnError),
                  (dict(workspace=torch.empty(9, dtype=torch.uint8, device="cuda")), ap.AttnError),
                  (dict(q=q[:, :3]), ap.AttnError)):
        with pytest.raises(e):
            f(**kw)
    o = torch.zeros_like(q)
    b = lambda **kw: ap.attn_bwd_packed(**{**dict(q=q, k=k, v=v, o=o, lse=lse, dout=do, cu_q=c, causal=True,  # noqa: E731
                                                  scale=0.1), **kw})
    for kw, e in ((dict(dout=do[:9]), ValueError), (dict(lse=lse.T), TypeError), (dict(o=o.float()), TypeError),
                  (dict(out=(q, k)), ValueError), (dict(out=(o, torch.zeros_like(k), torch.zeros_like(q))), ValueError),
                  (dict(workspace=torch.empty(9, dtype=torch.uint8, device="cuda")), ap.AttnError)):
        with pytest.raises(e):
            b(**kw)
    cos, sin = tables(50, 32)
    pos = torch.zeros(2, 80, dtype=torch.int32, device="cuda")
    r = lambda **kw: ap.rope_packed(**{**dict(q=q, k=k, positions=pos, cos=cos, sin=sin, sections=(10, 22)), **kw})  # noqa: E731
    for kw, e in ((dict(positions=pos.long()), TypeError), (dict(positions=pos[:, :5]), TypeError),
                  (dict(sections=(10, 23)), ValueError), (dict(sections=(32,)), ValueError), (dict(sections=(0, 32)), ValueError),
                  (dict(sin=sin[:9]), TypeError), (dict(cos=cos.double()), TypeError), (dict(k=k[:9]), ValueError),
                  (dict(out=(q, None)), ValueError), (dict(out=(q[:9], k)), ValueError), (dict(sections=None), ValueError)):
        with pytest.raises(e):
            r(**kw)
