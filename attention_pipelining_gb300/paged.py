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

import functools
import struct

from . import AttnError, _check, _load

# attn_kv_cache_t: k, v, block_table, format, num_pages, page_size, max_blocks, B, H_kv, D
_CACHE = struct.Struct("@PPPiiiiiii")
# attn_bhsd_t: data and the strides of the batch, the heads and the tokens
_BHSD = struct.Struct("@Pqqq")
KV_BF16, KV_INT4 = 0, 1
_INT_MAX = 2 ** 31 - 1   # the C entries' sizes are ints

# The checks below cost more than a small call's kernel if each goes through
# torch's slower accessors, so a call looks at each tensor once, and what is
# wrong is worked out only when something is.


torch = None   # imported with the first call, as in the package's other functions


def _import():
    global torch, _Tensor, _bf16, _u8, _i32, _f32, _current_device, _current_stream, _alloc, _free
    import torch as t
    _Tensor, _bf16, _u8, _i32, _f32 = t.Tensor, t.bfloat16, t.uint8, t.int32, t.float32
    _current_device, _current_stream, _alloc, _free = _short_ways(t._C)
    torch = t


def _short_ways(c):
    """The current device, its current stream's handle, and torch's caching allocator without a
    tensor around the memory (3 us less): by the functions behind torch.cuda's, which take a call
    less each, or by torch.cuda's own where a torch has no such name."""
    import torch.cuda as cuda
    return (getattr(c, "_cuda_getDevice", None) or cuda.current_device,
            getattr(c, "_cuda_getCurrentRawStream", None) or (
                lambda dev: cuda.current_stream(dev).cuda_stream),
            getattr(c, "_cuda_cudaCachingAllocator_raw_alloc", None) or (
                lambda nbytes, handle: cuda.caching_allocator_alloc(nbytes, stream=handle)),
            getattr(c, "_cuda_cudaCachingAllocator_raw_delete", None) or (
                cuda.caching_allocator_delete))


def _why_not_cache(k, v, bt):
    for name, t in (("k_cache", k), ("v_cache", v), ("block_table", bt)):
        if not isinstance(t, _Tensor) or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous CUDA tensor")
    if k.dtype not in (_bf16, _u8):
        raise TypeError("k_cache must be bfloat16 or, for a 4-bit cache, uint8")
    if bt.dtype != _i32 or bt.dim() != 2:
        raise TypeError("block_table must be an int32 [B, max_blocks] tensor")
    if v.device != k.device or bt.device != k.device:
        raise ValueError("k_cache, v_cache and block_table must be on one device")
    if k.dim() != 4 or v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError("k_cache and v_cache must be 4-D, of the same type and shape")
    raise ValueError("a 4-bit cache is [num_pages, H_kv, page_size / 16, 9 D]")


def _cache(k, v, bt):
    """(attn_kv_cache_t, device index, B, H_kv, D, positions the block table spans)"""
    if torch is None:
        _import()
    try:
        dev, dtype, shape = k.get_device(), k.dtype, k.shape
        if dev < 0 or v.get_device() != dev or bt.get_device() != dev or v.dtype is not dtype \
                or bt.dtype is not _i32 or v.shape != shape or not k.is_contiguous() \
                or not v.is_contiguous() or not bt.is_contiguous():
            raise ValueError
        pages, heads, page, D = shape
        B, blocks = bt.shape
        if dtype is _bf16:
            fmt = KV_BF16
        elif dtype is _u8 and D % 9 == 0:
            fmt, page, D = KV_INT4, 16 * page, D // 9
        else:
            raise ValueError
    except (ValueError, AttributeError):
        _why_not_cache(k, v, bt)
    return (_CACHE.pack(k.data_ptr(), v.data_ptr(), bt.data_ptr(), fmt, pages, page, blocks, B,
                        heads, D), dev, B, heads, D, blocks * page)


def _bhsd(name, t, shape, dev):
    """attn_bhsd_t of a bf16 tensor of that shape"""
    if not isinstance(t, _Tensor) or t.get_device() != dev or t.dtype is not _bf16:
        raise TypeError(f"{name} must be a bfloat16 tensor on the cache's device")
    sb, sh, ss, sd = t.stride() if t.shape == shape else (0, 0, 0, 0)
    if sd != 1:
        raise ValueError(f"{name} must be {list(shape)} with a contiguous last dimension, not "
                         f"{list(t.shape)} with strides {t.stride()}")
    return _BHSD.pack(t.data_ptr(), sb, sh, ss)


def _ints(name, t, B, dev, optional=False):
    if t is None and optional:
        return None
    if not isinstance(t, _Tensor) or t.get_device() != dev or t.dtype is not _i32 \
            or t.shape != (B,) or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 [{B}] tensor on the cache's device")
    return t.data_ptr()


def _out(name, t, shape, dtype, dev):
    if not isinstance(t, _Tensor) or t.get_device() != dev or t.dtype is not dtype \
            or t.shape != shape or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on the cache's "
                        "device")
    return t.data_ptr()


def _on(dev, stream, call):
    """call(stream handle) with device `dev` current, on `stream` or else on the device's current
    stream, to which what it allocates belongs."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("stream belongs to another device than the cache")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)
    if _current_device() == dev:
        return call(_current_stream(dev))
    with torch.cuda.device(dev):
        return call(_current_stream(dev))


def kv_cache_empty(num_pages: int, H_kv: int, page_size: int, D: int, fmt: str = "bf16",
                   device="cuda"):
    """A pair of uninitialised pools (k_cache, v_cache); fmt "bf16" or "int4"."""
    if torch is None:
        _import()
    if fmt not in ("bf16", "int4"):
        raise ValueError('fmt must be "bf16" or "int4"')
    if D not in (64, 128) or page_size <= 0 or page_size % 16:
        raise ValueError("D must be 64 or 128 and page_size a multiple of 16")
    shape = (num_pages, H_kv, page_size, D) if fmt == "bf16" else \
        (num_pages, H_kv, page_size // 16, 9 * D)
    dtype = _bf16 if fmt == "bf16" else _u8
    return (torch.empty(shape, dtype=dtype, device=device),
            torch.empty(shape, dtype=dtype, device=device))


def kv_append(k, v, k_cache, v_cache, block_table, start, cos=None, sin=None, q=None, q_out=None,
              new_lens=None, interleaved: bool = False, stream=None):
    """Writes new tokens k, v [B, H_kv, S, D] at positions start[b], start[b] + 1, .. of the cache,
    keys rotated by cos, sin [positions, rot_dim / 2] (float32; none: not rotated); with ``q``
    [B, H_q, S, D] also rotates the queries and returns them (in ``q_out`` if given, which may be q
    itself where q is contiguous; where new_lens leaves padding its rows keep what they held, zeros
    in a q_out allocated here)."""
    c, dev, B, heads, D, _ = _cache(k_cache, v_cache, block_table)
    if not isinstance(k, _Tensor) or k.dim() != 4:
        raise TypeError("k must be a [B, H_kv, S, D] tensor")
    S = k.shape[2]
    if S > _INT_MAX:   # (a view may claim any number of tokens)
        raise ValueError("S must be below 2^31")
    ks, vs = _bhsd("k", k, (B, heads, S, D), dev), _bhsd("v", v, (B, heads, S, D), dev)
    start_p, new_p = _ints("start", start, B, dev), _ints("new_lens", new_lens, B, dev, True)
    rows = rot = 0
    cos_p = sin_p = None
    if cos is not None or sin is not None:
        for name, t in (("cos", cos), ("sin", sin)):
            if not isinstance(t, _Tensor) or t.get_device() != dev or t.dtype is not _f32 \
                    or t.dim() != 2 or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous float32 [positions, rot_dim / 2] tensor "
                                "on the cache's device")
        if cos.shape != sin.shape or cos.shape[1] == 0:
            raise ValueError("cos and sin must have the same shape, with a rotation in them")
        rows, rot = cos.shape
        rot *= 2
        cos_p, sin_p = cos.data_ptr(), sin.data_ptr()
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
        H_q, qs = 0, None
    else:
        if not isinstance(q, _Tensor) or q.dim() != 4:
            raise TypeError("q must be a [B, H_q, S, D] tensor")
        H_q = q.shape[1]
        qs = _bhsd("q", q, (B, H_q, S, D), dev)

    def call(handle):
        out, out_p = q_out, None
        if q is not None:
            if out is None:
                make = torch.zeros if new_lens is not None else torch.empty
                out = make((B, H_q, S, D), dtype=_bf16, device=q.device)
            out_p = _out("q_out", out, (B, H_q, S, D), _bf16, dev)
        _check(_load().attn_kv_append(c, qs, out_p, ks, vs, start_p, new_p, cos_p, sin_p, rows, rot,
                                      1 if interleaved else 0, H_q, S, handle), "attn_kv_append")
        return out

    return _on(dev, stream, call)


def kv_read(k_cache, v_cache, block_table, lens, S: int, start=None, out=None, stream=None):
    """Positions start[b] .. start[b] + S - 1 (from 0 without ``start``) of every sequence as
    contiguous bf16 (k, v) [B, H_kv, S, D]; rows at or beyond lens[b] keep what ``out`` held, zeros
    where it is allocated here."""
    c, dev, B, heads, D, _ = _cache(k_cache, v_cache, block_table)
    lens_p, start_p = _ints("lens", lens, B, dev), _ints("start", start, B, dev, True)
    shape = (B, heads, S, D)

    def call(handle):
        k, v = out if out is not None else (
            torch.zeros(shape, dtype=_bf16, device=k_cache.device) for _ in range(2))
        _check(_load().attn_kv_read(c, _out("out[0]", k, shape, _bf16, dev),
                                    _out("out[1]", v, shape, _bf16, dev), lens_p, start_p, S, handle),
               "attn_kv_read")
        return k, v

    return _on(dev, stream, call)


@functools.lru_cache(maxsize=1024)
def paged_workspace_bytes(B, H_q, H_kv, S_q, D, max_keys) -> int:
    """Workspace bytes of attn_fwd_paged; max_keys: max_blocks * page_size."""
    return int(_load().attn_paged_workspace_bytes(B, H_q, H_kv, S_q, D, max_keys))


def attn_fwd_paged(q, k_cache, v_cache, block_table, lens, causal: bool, scale: float, q_lens=None,
                   workspace=None, out=None, stream=None, _fault=None):
    """Attention of q [B, H_q, S_q, D] over the first lens[b] cached positions of each sequence;
    returns (o, lse).  With ``causal`` the queries are the newest tokens (the last q_lens[b], or
    S_q, of lens[b]).  ``workspace``: optional uint8 tensor of at least paged_workspace_bytes(...)
    bytes, not shared with calls that may run at the same time (allocated if None); ``out``: optional
    (o, lse) to write into (rows of queries at or beyond q_lens[b] keep what it held, zeros where it
    is allocated here)."""
    c, dev, B, heads, D, span = _cache(k_cache, v_cache, block_table)
    if not isinstance(q, _Tensor) or q.dim() != 4:
        raise TypeError("q must be a [B, H_q, S_q, D] tensor")
    H_q, S_q = q.shape[1], q.shape[2]
    shape = (B, H_q, S_q, D)
    qs = _bhsd("q", q, shape, dev)
    lens_p, ql_p = _ints("lens", lens, B, dev), _ints("q_lens", q_lens, B, dev, True)
    nbytes = paged_workspace_bytes(B, H_q, heads, S_q, D, span)
    if nbytes == 0:
        raise AttnError(1, "attn_paged_workspace_bytes")
    if workspace is not None and (not isinstance(workspace, _Tensor)
                                  or workspace.get_device() != dev or workspace.dtype is not _u8
                                  or not workspace.is_contiguous()):
        raise TypeError("workspace must be a contiguous uint8 tensor on the cache's device")

    def call(handle):
        if out is None:
            make = torch.zeros if q_lens is not None else torch.empty
            o = make(shape, dtype=_bf16, device=q.device)
            lse = make(shape[:3], dtype=_f32, device=q.device)
        else:
            o, lse = out
        o_p, lse_p = _out("out[0]", o, shape, _bf16, dev), _out("out[1]", lse, shape[:3], _f32, dev)
        ws_p, ws_n, mine = None, 0, None
        if workspace is not None:
            ws_p, ws_n = workspace.data_ptr(), workspace.numel()
        elif nbytes > 256:   # 256: none is used
            ws_p = mine = _alloc(nbytes, handle)
            ws_n = nbytes
        try:
            args = (c, qs, o_p, lse_p, lens_p, ql_p, ws_p, ws_n, H_q, S_q, 1 if causal else 0, scale)
            if _fault is None:
                _check(_load().attn_fwd_paged(*args, handle), "attn_fwd_paged")
            else:
                _check(_load().attn_fwd_paged_timeout_test(*args, *_fault, handle),
                       "attn_fwd_paged_timeout_test")
        finally:
            if mine is not None:   # (used again only by what follows on the stream)
                _free(mine)
        return o, lse

    return _on(dev, stream, call)


def fwd_paged_timeout_test(q, k_cache, v_cache, block_table, lens, causal: bool, scale: float,
                           drop_stage: int, wait_budget_ns: int = 20_000_000, **kw):
    """Test hook: attn_fwd_paged with one stage of keys and values never requested, so that the
    kernel's bounded wait for it runs out (see attn_testing.h).  The device status word then reads
    ATTN_ERR_TIMEOUT."""
    return attn_fwd_paged(q, k_cache, v_cache, block_table, lens, causal, scale,
                          _fault=(int(drop_stage), int(wait_budget_ns)), **kw)
