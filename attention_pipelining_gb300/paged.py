"""The paged key/value cache and the attention that reads it (include/attn_paged.h).

    k_cache, v_cache = kv_cache_empty(num_pages, H_kv, page_size, D, "int4")
    q = kv_append(k, v, k_cache, v_cache, block_table, start, cos=cos, sin=sin, q=q)
    o, lse = attn_fwd_paged(q, k_cache, v_cache, block_table, lens, True, scale)
    k, v = kv_read(k_cache, v_cache, block_table, lens, S)

Argument marshalling only, as in the package's other entry points.  A bf16
cache is a pair of [num_pages, H_kv, page_size, D] tensors, a 4-bit cache a
pair of uint8 [num_pages, H_kv, page_size / 16, 9 D] tensors; the format and
the sizes follow from them.  ``block_table`` is int32 [B, max_blocks];
``lens``, ``start``, ``new_lens`` and ``q_lens`` are int32 [B]; all on the cache's
device.  q, k and v may have any strides that are multiples of 8 elements
with the last dimension contiguous.  Calls run on ``stream``, or else on the
current stream of the cache's device, whichever device is current; what they
allocate belongs to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes

from . import AttnError, _check, _load

KV_BF16, KV_INT4 = 0, 1


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("format", ctypes.c_int), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_blocks", ctypes.c_int), ("B", ctypes.c_int), ("H_kv", ctypes.c_int),
                ("D", ctypes.c_int)]


class _Bhsd(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64),
                ("stride_h", ctypes.c_int64), ("stride_s", ctypes.c_int64)]


def _cache(k_cache, v_cache, block_table):
    import torch
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("block_table", block_table)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous CUDA tensor")
    if k_cache.dtype == torch.bfloat16:
        fmt = KV_BF16
    elif k_cache.dtype == torch.uint8:
        fmt = KV_INT4
    else:
        raise TypeError("k_cache must be bfloat16 or, for a 4-bit cache, uint8")
    if k_cache.dim() != 4 or v_cache.dtype != k_cache.dtype or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be 4-D, of the same type and shape")
    if block_table.dtype != torch.int32 or block_table.dim() != 2:
        raise TypeError("block_table must be an int32 [B, max_blocks] tensor")
    if v_cache.device != k_cache.device or block_table.device != k_cache.device:
        raise ValueError("k_cache, v_cache and block_table must be on one device")
    pages, H_kv, page, D = k_cache.shape
    if fmt == KV_INT4:
        if D % 9:
            raise ValueError("a 4-bit cache is [num_pages, H_kv, page_size / 16, 9 D]")
        page, D = 16 * page, D // 9
    B, blocks = block_table.shape
    return _Cache(k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), fmt, pages, page,
                  blocks, B, H_kv, D)


def _bhsd(name, t, B, H, S, D, device):
    import torch
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be a bfloat16 tensor on the cache's device")
    if tuple(t.shape) != (B, H, S, D) or t.stride(3) != 1:
        raise ValueError(f"{name} must be [{B}, {H}, {S}, {D}] with a contiguous last dimension, "
                         f"not {tuple(t.shape)} with strides {tuple(t.stride())}")
    sb, sh, ss, _ = t.stride()
    return _Bhsd(t.data_ptr(), sb, sh, ss)


def _ints(name, t, B, device, optional=False):
    import torch
    if t is None and optional:
        return None
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.int32 \
            or tuple(t.shape) != (B,) or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 [{B}] tensor on the cache's device")
    return t.data_ptr()


def _out(name, t, shape, dtype, device):
    import torch
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != dtype \
            or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on the cache's device")
    return t


@contextlib.contextmanager
def _on(device, stream):
    """The device current and the stream's handle; what is allocated belongs to the stream."""
    import torch
    if stream is None:
        if torch.cuda.current_device() == device.index:
            yield torch.cuda.current_stream().cuda_stream
            return
        with torch.cuda.device(device):
            yield torch.cuda.current_stream(device).cuda_stream
        return
    if stream.device != device:
        raise ValueError("stream belongs to another device than the cache")
    with torch.cuda.stream(stream):
        yield stream.cuda_stream


def kv_cache_empty(num_pages: int, H_kv: int, page_size: int, D: int, fmt: str = "bf16",
                   device="cuda"):
    """A pair of uninitialised pools (k_cache, v_cache); fmt "bf16" or "int4"."""
    import torch
    if fmt not in ("bf16", "int4"):
        raise ValueError('fmt must be "bf16" or "int4"')
    if D not in (64, 128) or page_size <= 0 or page_size % 16:
        raise ValueError("D must be 64 or 128 and page_size a multiple of 16")
    shape = (num_pages, H_kv, page_size, D) if fmt == "bf16" else \
        (num_pages, H_kv, page_size // 16, 9 * D)
    dtype = torch.bfloat16 if fmt == "bf16" else torch.uint8
    return (torch.empty(shape, dtype=dtype, device=device),
            torch.empty(shape, dtype=dtype, device=device))


def kv_append(k, v, k_cache, v_cache, block_table, start, cos=None, sin=None, q=None, q_out=None,
              new_lens=None, interleaved: bool = False, stream=None):
    """Writes new tokens k, v [B, H_kv, S, D] at positions start[b], start[b] + 1, .. of the cache,
    keys rotated by cos, sin [positions, rot_dim / 2] (float32; none: not rotated); with ``q``
    [B, H_q, S, D] also rotates the queries and returns them (in ``q_out`` if given, which may be q
    itself where q is contiguous; where new_lens leaves padding its rows keep what they held, zeros
    in a q_out allocated here)."""
    import torch
    c = _cache(k_cache, v_cache, block_table)
    dev = k_cache.device
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise TypeError("k must be a [B, H_kv, S, D] tensor")
    S = k.shape[2]
    ks, vs = (_bhsd(n, t, c.B, c.H_kv, S, c.D, dev) for n, t in (("k", k), ("v", v)))
    start_p, new_p = _ints("start", start, c.B, dev), _ints("new_lens", new_lens, c.B, dev, True)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    rows = rot = 0
    cos_p = sin_p = None
    if cos is not None:
        for name, t in (("cos", cos), ("sin", sin)):
            if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != torch.float32 \
                    or t.dim() != 2 or not t.is_contiguous() or t.shape != cos.shape:
                raise TypeError(f"{name} must be a contiguous float32 [positions, rot_dim / 2] tensor "
                                "on the cache's device")
        rows, rot = cos.shape[0], 2 * cos.shape[1]
        cos_p, sin_p = cos.data_ptr(), sin.data_ptr()
        if rot == 0:
            raise ValueError("cos and sin hold no rotation")
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    with _on(dev, stream) as handle:
        H_q, qs, qo_p = 0, None, None
        if q is not None:
            if not isinstance(q, torch.Tensor) or q.dim() != 4:
                raise TypeError("q must be a [B, H_q, S, D] tensor")
            H_q = q.shape[1]
            qs = ctypes.byref(_bhsd("q", q, c.B, H_q, S, c.D, dev))
            if q_out is None:
                make = torch.zeros if new_lens is not None else torch.empty
                q_out = make((c.B, H_q, S, c.D), dtype=torch.bfloat16, device=dev)
            qo_p = _out("q_out", q_out, (c.B, H_q, S, c.D), torch.bfloat16, dev).data_ptr()
        _check(_load().attn_kv_append(ctypes.byref(c), qs, qo_p, ctypes.byref(ks), ctypes.byref(vs),
                                      start_p, new_p, cos_p, sin_p, rows, rot,
                                      int(bool(interleaved)), H_q, S, handle), "attn_kv_append")
    return q_out


def kv_read(k_cache, v_cache, block_table, lens, S: int, start=None, out=None, stream=None):
    """Positions start[b] .. start[b] + S - 1 (from 0 without ``start``) of every sequence as
    contiguous bf16 (k, v) [B, H_kv, S, D]; rows at or beyond lens[b] keep what ``out`` held, zeros
    where it is allocated here."""
    import torch
    c = _cache(k_cache, v_cache, block_table)
    dev = k_cache.device
    lens_p, start_p = _ints("lens", lens, c.B, dev), _ints("start", start, c.B, dev, True)
    shape = (c.B, c.H_kv, S, c.D)
    with _on(dev, stream) as handle:
        if out is None:
            out = tuple(torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
        k, v = (_out(n, t, shape, torch.bfloat16, dev) for n, t in zip(("out[0]", "out[1]"), out))
        _check(_load().attn_kv_read(ctypes.byref(c), k.data_ptr(), v.data_ptr(), lens_p, start_p, S,
                                    handle), "attn_kv_read")
    return k, v


def paged_workspace_bytes(B, H_q, H_kv, S_q, D) -> int:
    return int(_load().attn_paged_workspace_bytes(B, H_q, H_kv, S_q, D))


def attn_fwd_paged(q, k_cache, v_cache, block_table, lens, causal: bool, scale: float, q_lens=None,
                   workspace=None, out=None, stream=None):
    """Attention of q [B, H_q, S_q, D] over the first lens[b] cached positions of each sequence;
    returns (o, lse).  With ``causal`` the queries are the newest tokens (the last q_lens[b], or
    S_q, of lens[b]).  ``workspace``: optional uint8 tensor of at least paged_workspace_bytes(...)
    bytes, not shared with calls that may run at the same time (allocated if None); ``out``: optional
    (o, lse) to write into (rows of queries at or beyond q_lens[b] keep what it held, zeros where it
    is allocated here)."""
    import torch
    c = _cache(k_cache, v_cache, block_table)
    dev = k_cache.device
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise TypeError("q must be a [B, H_q, S_q, D] tensor")
    H_q, S_q = q.shape[1], q.shape[2]
    qs = _bhsd("q", q, c.B, H_q, S_q, c.D, dev)
    lens_p, ql_p = _ints("lens", lens, c.B, dev), _ints("q_lens", q_lens, c.B, dev, True)
    lib = _load()
    nbytes = int(lib.attn_paged_workspace_bytes(c.B, H_q, c.H_kv, S_q, c.D))
    if nbytes == 0:
        raise AttnError(1, "attn_paged_workspace_bytes")
    with _on(dev, stream) as handle:
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        elif not isinstance(workspace, torch.Tensor) or workspace.device != dev \
                or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous uint8 tensor on the cache's device")
        if out is None:
            make = torch.zeros if q_lens is not None else torch.empty
            out = (make((c.B, H_q, S_q, c.D), dtype=torch.bfloat16, device=dev),
                   make((c.B, H_q, S_q), dtype=torch.float32, device=dev))
        o = _out("out[0]", out[0], (c.B, H_q, S_q, c.D), torch.bfloat16, dev)
        lse = _out("out[1]", out[1], (c.B, H_q, S_q), torch.float32, dev)
        _check(lib.attn_fwd_paged(ctypes.byref(c), ctypes.byref(qs), o.data_ptr(), lse.data_ptr(),
                                  lens_p, ql_p, workspace.data_ptr(), workspace.numel(), H_q, S_q,
                                  int(bool(causal)), float(scale), handle), "attn_fwd_paged")
    return o, lse
