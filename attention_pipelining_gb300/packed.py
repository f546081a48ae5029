"""Packed sequences: rotation with several axes, attention and its gradients (include/attn_packed.h).

    q, k = rope_packed(q, k, positions, cos, sin, sections)
    o, lse = attn_fwd_packed(q, k, v, cu, True, scale)
    dq, dk, dv = attn_bwd_packed(q, k, v, o, lse, dout, cu, True, scale)
    dq, dk = rope_packed(dq, dk, positions, cos, sin, sections, inverse=True, out=(dq, dk))

Argument marshalling only, as in the package's other entry points.  The tokens of all sequences lie
one after the other: q [T, H_q, D], k and v [T, H_kv, D] bf16, and ``cu`` int32 [B + 1] says where
they begin and end (sequence b is tokens cu[b] .. cu[b + 1] - 1; any may be empty).  With ``cu_k`` the
keys have lengths, and a number of tokens, of their own.  Tensors may have any positive strides that
are multiples of 8 elements with the last dimension contiguous (views of one projection's output).
Calls run on ``stream``, or else on the current stream of the tensors' device, whichever device is
current; what they allocate belongs to that stream.
"""
from __future__ import annotations

import functools
import struct

from . import _check, _load, paged

# attn_packed_t: B, T_q, T_k, H_q, H_kv, D, causal, scale
_SIZES = struct.Struct("@iiiiiiif")
# attn_thd_t: data and the strides of the tokens and the heads
_THD = struct.Struct("@Pqq")
_INT_MAX = 2 ** 31 - 1   # the C entries' sizes are ints

torch = None   # imported with the first call, as in the package's other functions


def _import():
    global torch, _Tensor, _bf16, _u8, _i32, _f32, _alloc, _free
    if paged.torch is None:
        paged._import()
    _Tensor, _bf16, _u8, _i32, _f32 = paged._Tensor, paged._bf16, paged._u8, paged._i32, paged._f32
    _alloc, _free = paged._alloc, paged._free
    torch = paged.torch


# A call looks at each tensor once, and what is wrong is worked out only when something is: a small
# call's kernels take less time than torch's accessors.


def _device(name, t):
    """The device index of a call's first tensor"""
    if torch is None:
        _import()
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a bfloat16 CUDA tensor [tokens, heads, D]")
    return t.get_device()


def _thd(name, t, dev):
    """(attn_thd_t, shape) of a bf16 tensor [tokens, heads, D]"""
    try:
        st, sh, sd = t.stride()
        if sd == 1 and t.dtype is _bf16 and t.get_device() == dev:
            return _THD.pack(t.data_ptr(), st, sh), t.shape
    except (AttributeError, TypeError, ValueError):
        pass
    if not isinstance(t, _Tensor) or t.get_device() != dev or t.dtype is not _bf16 or t.dim() != 3:
        raise TypeError(f"{name} must be a bfloat16 tensor [tokens, heads, D] on the same device as the others")
    raise ValueError(f"{name}'s last dimension must be contiguous, not with strides {t.stride()}")


def _like(name, t, shape, dev):
    """attn_thd_t of a bf16 tensor of that shape"""
    x, got = _thd(name, t, dev)
    if got != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(got)}")
    return x


def _flat(name, t, shape, dtype, dev):
    try:
        if t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except (AttributeError, TypeError):
        pass
    raise TypeError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on the same device as the others")


def _small(*sizes):
    if max(sizes) > _INT_MAX:   # (a view may claim any number of tokens)
        raise ValueError("sizes must be below 2^31")


def _sizes(q, k, v, cu_q, cu_k, causal, scale):
    """What both attention calls begin with: device, shapes, attn_packed_t, tensors and bounds."""
    dev = _device("q", q)
    (qs, q_shape), (ks, k_shape), (vs, v_shape) = _thd("q", q, dev), _thd("k", k, dev), _thd("v", v, dev)
    T_q, H_q, D = q_shape
    T_k, H_kv, Dk = k_shape
    if k_shape != v_shape or D != Dk or (cu_k is None and T_k != T_q):
        raise ValueError(f"q {list(q_shape)}, k {list(k_shape)} and v {list(v_shape)} do not go together"
                         + ("" if cu_k is not None else " (without cu_k they have the same tokens)"))
    if not isinstance(cu_q, _Tensor) or cu_q.dim() != 1 or cu_q.shape[0] < 2:
        raise TypeError("cu_q must be an int32 [sequences + 1] tensor")
    bounds = cu_q.shape
    B = bounds[0] - 1
    _small(T_q, T_k, H_q, H_kv, D, B)
    return (dev, q_shape, k_shape, _SIZES.pack(B, T_q, T_k, H_q, H_kv, D, 1 if causal else 0, scale), qs, ks, vs,
            _flat("cu_q", cu_q, bounds, _i32, dev),
            None if cu_k is None else _flat("cu_k", cu_k, bounds, _i32, dev))


@functools.lru_cache(maxsize=1024)
def _fwd_bytes(sizes) -> int:
    return int(_load().attn_packed_workspace_bytes(sizes))


@functools.lru_cache(maxsize=1024)
def _bwd_bytes(sizes, deterministic) -> int:
    return int(_load().attn_packed_bwd_workspace_bytes(sizes, deterministic))


def packed_workspace_bytes(B: int, T_q: int, T_k: int, H_q: int, H_kv: int, D: int) -> int:
    """Workspace bytes of attn_fwd_packed (0 if the sizes are invalid)."""
    return _fwd_bytes(_SIZES.pack(B, T_q, T_k, H_q, H_kv, D, 0, 1.0))


def packed_bwd_workspace_bytes(B: int, T_q: int, T_k: int, H_q: int, H_kv: int, D: int,
                               deterministic: bool = False) -> int:
    """Workspace bytes of attn_bwd_packed (0 if the sizes are invalid)."""
    return _bwd_bytes(_SIZES.pack(B, T_q, T_k, H_q, H_kv, D, 0, 1.0), 1 if deterministic else 0)


def _given(workspace, dev):
    """(pointer, bytes) of a caller's workspace"""
    if not isinstance(workspace, _Tensor) or workspace.get_device() != dev \
            or workspace.dtype is not _u8 or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor on the same device as the others")
    return workspace.data_ptr(), workspace.numel()


def attn_fwd_packed(q, k, v, cu_q, causal: bool, scale: float, cu_k=None, workspace=None, out=None,
                    stream=None, _fault=None):
    """Attention of every sequence over its own keys; returns (o [T_q, H_q, D] bf16, lse [H_q, T_q]
    float32).  With ``causal`` the queries are the newest of the sequence's tokens: of n queries and m
    keys query i sees keys j <= i + m - n.  ``workspace``: optional uint8 tensor of at least
    packed_workspace_bytes(...) bytes, not shared with calls that may run at the same time (allocated
    if None); ``out``: optional (o, lse) to write into (rows of tokens that belong to no sequence keep
    what it held, zeros where it is allocated here)."""
    # (the tensors keep their names: a caller may hold no other reference to one, and what is free
    # the workspace may get)
    dev, q_shape, k_shape, sizes, qs, ks, vs, cq, ck = _sizes(q, k, v, cu_q, cu_k, causal, scale)
    lse_shape = (q_shape[1], q_shape[0])
    nbytes = _fwd_bytes(sizes)
    if nbytes == 0:   # (refused: the entry looks at the sizes first, and says why)
        _check(_load().attn_fwd_packed(sizes, *[None] * 8, 0, None), "attn_fwd_packed")

    def call(handle):
        o, lse = out if out is not None else (
            torch.zeros(q_shape, dtype=_bf16, device=q.device),
            torch.zeros(lse_shape, dtype=_f32, device=q.device))
        os, lse_p = _like("out[0]", o, q_shape, dev), _flat("out[1]", lse, lse_shape, _f32, dev)
        ws, n = _given(workspace, dev) if workspace is not None else (_alloc(nbytes, handle), nbytes)
        try:
            args = (sizes, qs, ks, vs, os, lse_p, cq, ck, ws, n)
            if _fault is None:
                _check(_load().attn_fwd_packed(*args, handle), "attn_fwd_packed")
            else:
                _check(_load().attn_fwd_packed_timeout_test(*args, *_fault, handle),
                       "attn_fwd_packed_timeout_test")
        finally:   # (used again only by what follows on the stream)
            if workspace is None:
                _free(ws)
        return o, lse

    return paged._on(dev, stream, call)


def attn_bwd_packed(q, k, v, o, lse, dout, cu_q, causal: bool, scale: float, cu_k=None, workspace=None,
                    out=None, deterministic: bool = False, stream=None, _fault=None):
    """Gradients (dq, dk, dv) of attn_fwd_packed's q, k and v for the gradient ``dout`` of its o, given
    its o and lse.  ``workspace``: optional uint8 tensor of at least packed_bwd_workspace_bytes(...)
    bytes, not shared with calls that may run at the same time (allocated if None); ``out``: optional
    (dq, dk, dv) to write into (rows of tokens that belong to no sequence keep what it held, zeros
    where it is allocated here).  ``deterministic``: dq reproducible bit for bit (dk and dv always
    are)."""
    dev, q_shape, k_shape, sizes, qs, ks, vs, cq, ck = _sizes(q, k, v, cu_q, cu_k, causal, scale)
    os, dos = _like("o", o, q_shape, dev), _like("dout", dout, q_shape, dev)
    lse_p = _flat("lse", lse, (q_shape[1], q_shape[0]), _f32, dev)
    det = 1 if deterministic else 0
    nbytes = _bwd_bytes(sizes, det)
    if nbytes == 0:
        _check(_load().attn_bwd_packed(sizes, *[None] * 12, 0, det, None), "attn_bwd_packed")

    def call(handle):
        dq, dk, dv = out if out is not None else (
            torch.zeros(s, dtype=_bf16, device=q.device) for s in (q_shape, k_shape, k_shape))
        dqs, dks = _like("out[0]", dq, q_shape, dev), _like("out[1]", dk, k_shape, dev)
        dvs = _like("out[2]", dv, k_shape, dev)
        ws, n = _given(workspace, dev) if workspace is not None else (_alloc(nbytes, handle), nbytes)
        try:
            args = (sizes, qs, ks, vs, os, lse_p, dos, dqs, dks, dvs, cq, ck, ws, n, det)
            if _fault is None:
                _check(_load().attn_bwd_packed(*args, handle), "attn_bwd_packed")
            else:
                _check(_load().attn_bwd_packed_timeout_test(*args, *_fault, handle),
                       "attn_bwd_packed_timeout_test")
        finally:
            if workspace is None:
                _free(ws)
        return dq, dk, dv

    return paged._on(dev, stream, call)


def fwd_packed_timeout_test(*args, drop_block: int, wait_budget_ns: int = 20_000_000, **kw):
    """Test hook: attn_fwd_packed with one "P stored" signal withheld, so that the kernel's bounded
    wait for it runs out (see attn_testing.h).  The device status word then reads ATTN_ERR_TIMEOUT."""
    return attn_fwd_packed(*args, _fault=(int(drop_block), int(wait_budget_ns)), **kw)


def bwd_packed_timeout_test(*args, drop_item: int, wait_budget_ns: int = 20_000_000, **kw):
    """Test hook: attn_bwd_packed likewise, in its dK/dV kernel (and its dQ kernel, if deterministic)."""
    return attn_bwd_packed(*args, _fault=(int(drop_item), int(wait_budget_ns)), **kw)


@functools.lru_cache(maxsize=256)
def _sections(sections, axes, pairs):
    """The sections as the C entry takes them"""
    if sections is None:
        sections = (pairs,)
    if len(sections) != axes or sum(sections) != pairs or min(sections) <= 0:
        raise ValueError(f"sections must be {axes} positive numbers of pairs whose sum is {pairs}")
    return struct.pack(f"@{axes}i", *sections)


def rope_packed(q, k, positions, cos, sin, sections=None, interleaved: bool = False,
                inverse: bool = False, out=None, stream=None):
    """Rotates queries q [T, H_q, D] and keys k [T, H_kv, D] (either may be None) by positions with one
    to four axes and returns both.  ``positions`` int32 [axes, T]; ``cos`` and ``sin`` float32 [rows,
    rot_dim / 2], one row a position; the pairs of elements fall into ``sections`` (pairs of each axis,
    their sum rot_dim / 2; None with one axis: all of them).  ``inverse``: the other way round, which is
    the gradient's.  ``out``: optional (q, k) to write into, which may be q and k themselves.  A token with
    a position outside the tables is skipped (its output rows keep what ``out`` held, and are unspecified
    where it is allocated here) and recorded in the status word."""
    x = q if q is not None else k
    dev = _device("q" if q is not None else "k", x)
    qs = ks = q_shape = k_shape = None
    H_q = H_kv = 0
    if k is not None:
        ks, k_shape = _thd("k", k, dev)
        T, H_kv, D = k_shape
    if q is not None:
        qs, q_shape = _thd("q", q, dev)
        T, H_q, D = q_shape
        if k is not None and (T, D) != (k_shape[0], k_shape[2]):
            raise ValueError(f"q {list(q_shape)} and k {list(k_shape)} do not go together")
    if not isinstance(positions, _Tensor) or positions.dim() != 2 or not isinstance(cos, _Tensor) \
            or cos.dim() != 2:
        raise TypeError("positions must be an int32 [axes, T] tensor and cos a float32 [rows, rot_dim / 2] one")
    axes, table = positions.shape[0], cos.shape
    rows, pairs = table
    _small(T, H_q, H_kv, D, rows, 2 * pairs, axes)
    pos_p = _flat("positions", positions, (axes, T), _i32, dev)
    cos_p, sin_p = _flat("cos", cos, table, _f32, dev), _flat("sin", sin, table, _f32, dev)
    sections = _sections(None if sections is None else tuple(sections), axes, pairs)

    def call(handle):
        qo, ko = out if out is not None else (
            None if q is None else torch.empty(q_shape, dtype=_bf16, device=x.device),
            None if k is None else torch.empty(k_shape, dtype=_bf16, device=x.device))
        if (qo is None) != (q is None) or (ko is None) != (k is None):
            raise ValueError("out must have a tensor for each of q and k that there is")
        _check(_load().attn_rope_packed(
            qs, None if q is None else _like("out[0]", qo, q_shape, dev),
            ks, None if k is None else _like("out[1]", ko, k_shape, dev),
            pos_p, sections, axes, cos_p, sin_p, rows, 2 * pairs, 1 if interleaved else 0,
            1 if inverse else 0, T, H_q, H_kv, D, handle), "attn_rope_packed")
        return qo, ko

    return paged._on(dev, stream, call)
