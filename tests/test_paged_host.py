"""The paged cache's entry points refuse bad arguments on the host, before any CUDA
call (CPU only; fake, never-dereferenced device addresses)."""
import ctypes

import numpy as np
import pytest
import torch

import attention_pipelining_gb300 as ap
from attention_pipelining_gb300 import paged
from tests import paged_ref as ref

A = 0x10000


@pytest.fixture(scope="module")
def lib():
    ap.build()
    return ap._load()


def cache(**kw):
    d = dict(k=A, v=A, block_table=A, format=0, num_pages=10, page_size=64, max_blocks=8, B=2, H_kv=2,
             D=128)
    d.update(kw)
    return paged._CACHE.pack(*[d[n] or 0 for n in (
        "k", "v", "block_table", "format", "num_pages", "page_size", "max_blocks", "B", "H_kv", "D")])


def tensor(data=A, sb=8 * 128, sh=128, ss=2 * 128):
    return paged._BHSD.pack(data or 0, sb, sh, ss)


def append(lib, c=None, q=None, q_out=None, k=None, v=None, start=A, new=None, cos=A, sin=A,
           rows=512, rot=128, inter=0, H_q=0, S=4):
    c = cache() if c is None else c
    k, v = k or tensor(), v or tensor()
    return lib.attn_kv_append(c, q, q_out, k, v,
                              start, new, cos, sin, rows, rot, inter, H_q, S, None)


def read(lib, c=None, k=A, v=A, lens=A, start=None, S=4):
    c = cache() if c is None else c
    return lib.attn_kv_read(c, k, v, lens, start, S, None)


def attend(lib, c=None, q=None, o=A, lse=A, lens=A, q_lens=None, ws=A, nbytes=1 << 30, H_q=4,
           S_q=1, causal=1, scale=0.1):
    c = cache() if c is None else c
    q = q or tensor()
    return lib.attn_fwd_paged(c, q, o, lse, lens, q_lens, ws, nbytes,
                              H_q, S_q, causal, ctypes.c_float(scale), None)


BAD_CACHE = [(dict(k=None), 1), (dict(v=None), 1), (dict(block_table=None), 1), (dict(B=0), 1),
             (dict(H_kv=-1), 1), (dict(D=0), 1), (dict(num_pages=0), 1), (dict(page_size=0), 1),
             (dict(max_blocks=0), 1), (dict(format=2), 1), (dict(page_size=24), 1),
             (dict(D=96), 2), (dict(B=70000), 2), (dict(H_kv=40000), 2),
             (dict(max_blocks=1 << 24), 2), (dict(num_pages=2**31 - 1, H_kv=32767, page_size=4096), 2),
             (dict(k=A + 8), 3), (dict(v=A + 4), 3), (dict(block_table=A + 2), 3)]


@pytest.mark.parametrize("kw,code", BAD_CACHE, ids=[str(k) for k, _ in BAD_CACHE])
def test_every_entry_checks_the_cache(lib, kw, code):
    c = cache(**kw)
    assert append(lib, c) == code
    assert read(lib, c) == code
    assert attend(lib, c) == code


@pytest.mark.parametrize("kw,code", [
    (dict(start=None), 1), (dict(S=0), 1), (dict(H_q=-1), 1), (dict(H_q=2), 1),
    (dict(H_q=2, q=tensor()), 1), (dict(q=tensor(), q_out=A), 1), (dict(inter=2), 1),
    (dict(rot=-16), 1), (dict(rot=144), 1), (dict(rot=24), 1), (dict(cos=None), 1),
    (dict(sin=None), 1), (dict(rows=0), 1), (dict(S=1 << 30), 2), (dict(start=A + 2), 3),
    (dict(cos=A + 8), 3), (dict(k=tensor(data=None)), 1), (dict(k=tensor(A + 8)), 3),
    (dict(v=tensor(sb=12)), 3), (dict(k=tensor(sh=4)), 3), (dict(v=tensor(ss=129)), 3),
    (dict(H_q=2, q=tensor(A + 2), q_out=A), 3), (dict(H_q=2, q=tensor(), q_out=A + 8), 3),
    (dict(H_q=70000, q=tensor(), q_out=A), 2),
])
def test_append_refuses(lib, kw, code):
    assert append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(lens=None), 1), (dict(S=0), 1), (dict(S=-2), 1),
    (dict(S=1 << 30), 2), (dict(k=A + 8), 3), (dict(v=A + 2), 3), (dict(lens=A + 1), 3),
    (dict(start=A + 2), 3),
])
def test_read_refuses(lib, kw, code):
    assert read(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(o=None), 1), (dict(lse=None), 1), (dict(lens=None), 1),
    (dict(causal=2), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(H_q=3), 1), (dict(H_q=0), 1), (dict(S_q=0), 1), (dict(S_q=1 << 30), 2),
    (dict(q=tensor(data=None)), 1), (dict(q=tensor(sh=20)), 3), (dict(o=A + 8), 3),
    (dict(lse=A + 2), 3), (dict(ws=A + 16), 3), (dict(q_lens=A + 1), 3),
])
def test_attention_refuses(lib, kw, code):
    assert attend(lib, **kw) == code


@pytest.mark.parametrize("drop,budget,code", [(-1, 10**7, 1), (0, 999_999, 1), (0, 2**63, 1)])
def test_timeout_hook_refuses(lib, drop, budget, code):
    assert lib.attn_fwd_paged_timeout_test(cache(), tensor(), A, A, A, None, A, 1 << 30, 4, 1, 1,
                                           ctypes.c_float(0.1), drop, budget, None) == code


def test_attention_checks_the_workspace_of_split_items(lib):
    need = lib.attn_paged_workspace_bytes(2, 4, 2, 1, 128, 64 * 40)
    assert attend(lib, cache(max_blocks=40), nbytes=need - 1) == 1
    assert attend(lib, cache(max_blocks=40), ws=None) == 1
    assert attend(lib, cache(max_blocks=16), ws=None, nbytes=0, o=A + 8) == 3   # needs none
    assert attend(lib, cache(max_blocks=40), nbytes=need, o=A + 8) == 3   # stops at another rule


def test_strides_of_single_dimensions_are_not_looked_at(lib):
    """[B, 1, 1, D] views may carry any stride there: the call stops at a later rule."""
    c = cache(H_kv=1)
    odd = tensor(sh=3, ss=5)
    assert append(lib, c, k=odd, v=tensor(A + 2, sh=3, ss=5), S=1) == 3   # v's address, not k's strides
    assert append(lib, c, k=odd, v=tensor(A, sh=3, ss=5), S=1, rows=0) == 1


def test_workspace_bytes(lib):
    """Two parts of each of at most 512 thread blocks, D + 1 floats a row of the tile, and 16
    bytes a thread block; one block a unit of 64 keys where there are fewer units; next to
    nothing where the block tables span no more keys than an item is kept whole for."""
    f = lib.attn_paged_workspace_bytes
    for H_q, H_kv, S_q, rows in ((8, 1, 1, 8), (9, 1, 1, 16), (32, 8, 1, 8), (32, 8, 4, 16),
                                 (32, 8, 5, 32), (32, 8, 9, 64), (32, 8, 500, 64)):
        for D in (64, 128):
            assert f(300, H_q, H_kv, S_q, D, 4096) == 512 * (2 * rows * (D + 1) * 4 + 16)
            assert f(300, H_q, H_kv, S_q, D, 1024) == 256
    assert f(2, 8, 2, 1, 64, 1025) == 2 * 2 * 17 * (2 * 8 * 65 * 4 + 16)
    for bad in ((0, 8, 1, 1, 64, 9), (1, 8, 3, 1, 64, 9), (1, 8, 1, 0, 64, 9), (1, 8, 1, 1, 96, 9),
                (1, 8, 1, 1, 64, 0)):
        assert f(*bad) == 0


def test_binding_refuses_on_the_host():
    t = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    pool = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16)
    bt = torch.zeros(1, 4, dtype=torch.int32)
    n = torch.ones(1, dtype=torch.int32)
    for f in (lambda: ap.kv_append(t, t, pool, pool, bt, n),
              lambda: ap.kv_read(pool, pool, bt, n, 4),
              lambda: ap.attn_fwd_paged(t, pool, pool, bt, n, True, 0.1)):
        with pytest.raises(TypeError):   # not on a GPU
            f()
    for bad in (dict(fmt="fp8"), dict(D=80), dict(page_size=20), dict(page_size=0)):
        with pytest.raises(ValueError):
            ap.kv_cache_empty(**{**dict(num_pages=2, H_kv=1, page_size=16, D=64, device="cpu"), **bad})
    k, v = ap.kv_cache_empty(3, 2, 48, 128, "int4", device="cpu")
    assert k.shape == v.shape == (3, 2, 3, 9 * 128) and k.dtype == torch.uint8
    k, v = ap.kv_cache_empty(3, 2, 48, 64, device="cpu")
    assert k.shape == (3, 2, 48, 64) and k.dtype == torch.bfloat16


# ---------------------------------------------------------------- the reference itself


@pytest.mark.parametrize("kind", ["k", "v"])
@pytest.mark.parametrize("D", [64, 128])
def test_reference_format(kind, D):
    """Every nibble of a block belongs to one element, no byte to two tokens; packed
    values come back within half a step of their group, or as NaN."""
    idx = ref.nibble_index(kind, D)
    assert sorted(idx.ravel()) == list(range(16 * D))
    owner = np.zeros(16 * D, int)
    owner[idx] = np.arange(16)[:, None]
    assert (owner[0::2] == owner[1::2]).all()
    x = ref.bf16(np.random.default_rng(3).normal(size=(48, D)))
    x[5, :32] = 0.0
    x[7, 33] = np.inf
    y, s = ref.unpack(ref.pack(x, kind), kind)
    assert np.isnan(y[7, 32:64]).all() and (y[5, :32] == 0).all()
    e = np.abs(y - x).reshape(48, D // 32, 32)
    ok = np.isfinite(s)
    assert (e[ok] <= 0.5 * s[ok][:, None] * (1 + 2.0 ** -5)).all()


def test_reference_attention_matches_torch():
    """The reference on one sequence against torch's float64 softmax."""
    g = np.random.default_rng(4)
    vals = g.normal(size=(3, 2, 16, 64)), g.normal(size=(3, 2, 16, 64))
    q = g.normal(size=(1, 4, 2, 64))
    table = np.array([[2, 0]])
    o, lse, _, _ = ref.attention(q, *vals, None, None, table, [21], 16, True, 0.2)
    k, v = (torch.from_numpy(np.concatenate([x[2], x[0]], 1)[:, :21]) for x in vals)
    for h in range(4):
        for i in range(2):
            s = 0.2 * k[h // 2][:20 + i] @ torch.from_numpy(q[0, h, i])
            assert np.allclose(torch.softmax(s, 0) @ v[h // 2][:20 + i], o[0, h, i], atol=1e-12)
            assert np.allclose(torch.logsumexp(s, 0), lse[0, h, i], atol=1e-12)


def test_a_torch_without_the_short_ways(monkeypatch):
    """Where torch has no function of the names that the binding takes first, it takes
    torch.cuda's own."""
    class Stream:
        cuda_stream = 77
    calls = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: Stream)
    monkeypatch.setattr(torch.cuda, "caching_allocator_alloc",
                        lambda n, device=None, stream=None: calls.append((n, stream)) or 0x4000)
    monkeypatch.setattr(torch.cuda, "caching_allocator_delete", calls.append)
    device, stream, alloc, free = paged._short_ways(object())
    assert device() == 3 and stream(3) == 77
    assert alloc(512, 77) == 0x4000 and free(0x4000) is None
    assert calls == [(512, 77), 0x4000]
    # and the first ones where they are there
    class Names:
        _cuda_getDevice, _cuda_getCurrentRawStream = (lambda: 5), (lambda dev: dev + 1)
        _cuda_cudaCachingAllocator_raw_alloc, _cuda_cudaCachingAllocator_raw_delete = max, min
    got = paged._short_ways(Names)
    assert got[0]() == 5 and got[1](8) == 9 and got[2:] == (max, min)
