"""The paged cache and its operators in 64 bits (numpy), from the definitions of
include/attn_paged.h: the reference of tests/test_gpu_paged.py.

Also the error bounds of the CUDA attention, from its rounding model:

* O's rounding to bf16: 2^-8 of |O|.
* The rounding of the probabilities (to bf16 for a bf16 cache: 2^-8; times the
  values' scales to fp16 for a 4-bit one: 2^-11, and 2^-25 absolute below
  2^-14 where the largest product of the row's 16-key block is 2^5 or more).  O's error
  is that share of A = sum_j p_j |v_j| / sum_j p_j.
* The scores' error, which every probability takes as a relative error (twice in
  O: numerator and denominator): tensor-core sums in fp32, at most 2^-20 of the
  sum of the magnitudes per instruction chain (eight instructions of at most
  four steps of 2^-23 each at D = 128 give 2^-18); for 4-bit keys also a
  query's fp16 rounding of at most 2^-11 2^-14 of its row's largest element; then
  the exponent's three fp32 roundings (2^-22 of its magnitude) and ex2's 2^-22.
"""
import numpy as np
import torch


def bf16(x):
    """Nearest value with 8 significant bits (float64 arrays in bf16's normal range)."""
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.round(m * 256), e - 8)


def f64(t):
    return t.detach().cpu().double().numpy()


def to_bf16_tensor(x):
    """float64 values that are bf16 numbers (or the nearest ones) as a tensor."""
    return torch.from_numpy(bf16(x)).to(torch.bfloat16)


# ---------------------------------------------------------------- the 4-bit format


def quantise(x):
    """x [..., D] -> (codes 0 .. 15 [..., D] uint8, scales [..., D / 32] float64)."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(g).max(-1)
    ok = np.isfinite(amax)
    s = np.where(ok, bf16(np.where(ok, amax, 0.0) / 7), np.nan)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where((s > 0)[..., None], np.clip(np.round(g / s[..., None]), -7, 7), 0.0)
    return (q + 8).astype(np.uint8).reshape(x.shape), s


def nibble_index(kind, D):
    """[16, D]: in which nibble of a block (byte 2 i's low, high, ...) element d of token r is."""
    G = D // 32
    out = np.zeros((16, D), np.int64)
    for r in range(16):
        for d in range(D):
            j, e = d // 32, d % 32
            if kind == "k":
                out[r, d] = 2 * (r * D // 2 + ((e // 8) * G + j) * 4) + e % 8
            else:
                out[r, d] = 2 * ((((r // 2) * 8 + e // 4) * 2 + r % 2) * 2 * G + 2 * j) + e % 4
    return out


def pack(x, kind):
    """x [n, D] float64, n a multiple of 16 -> bytes [n / 16, 9 D]."""
    n, D = x.shape
    codes, s = quantise(x)
    nib = np.zeros((n // 16, 16 * D), np.uint8)
    idx = nibble_index(kind, D)
    nib[:, idx.ravel()] = codes.reshape(n // 16, 16 * D)
    sb = to_bf16_tensor(np.nan_to_num(s)).view(torch.int16).numpy().view(np.uint16)
    sb = np.where(np.isnan(s), np.uint16(0x7fff), sb).astype("<u2")
    return np.concatenate([nib[:, 0::2] | (nib[:, 1::2] << 4),
                           sb.reshape(n // 16, -1).view(np.uint8)], 1)


def unpack(blocks, kind):
    """bytes [m, 9 D] -> float64 values [16 m, D]."""
    m, n = blocks.shape
    D = n // 9
    nib = np.zeros((m, 16 * D), np.uint8)
    nib[:, 0::2], nib[:, 1::2] = blocks[:, :8 * D] & 15, blocks[:, :8 * D] >> 4
    c = nib[:, nibble_index(kind, D).ravel()].reshape(m * 16, D // 32, 32).astype(np.float64) - 8
    sb = np.ascontiguousarray(blocks[:, 8 * D:]).view(np.uint16).astype(np.uint32) << 16
    s = sb.view(np.float32).astype(np.float64).reshape(m * 16, D // 32, 1)
    return (c * s).reshape(m * 16, D), s[..., 0]


def cache_values(cache, kind):
    """A whole cache tensor as float64 [pages, H, page_size, D] and, for 4 bits, the scales."""
    c = cache.cpu()
    if c.dtype == torch.bfloat16:
        return c.double().numpy(), None
    P, H, m, n = c.shape
    v, s = unpack(c.numpy().reshape(-1, n), kind)
    D = n // 9
    return v.reshape(P, H, 16 * m, D), s.reshape(P, H, 16 * m, D // 32)


def gather(vals, table, n, page):
    """The first n positions [H, n, ...] of one sequence whose pages are table."""
    pages = table[:-(-n // page)] if n else table[:0]
    if n == 0:
        return vals[0][:, :0]
    x = np.concatenate([vals[p] for p in pages], 1)
    return x[:, :n]


# ---------------------------------------------------------------- operators


def rotate(x, cos, sin, interleaved):
    """x [..., S, D], cos and sin [..., S, rot / 2]; rounded to bf16."""
    rot = 2 * cos.shape[-1]
    y = np.array(x, np.float64)
    if interleaved:
        a, b = y[..., 0:rot:2].copy(), y[..., 1:rot:2].copy()
        y[..., 0:rot:2], y[..., 1:rot:2] = bf16(a * cos - b * sin), bf16(b * cos + a * sin)
    else:
        a, b = y[..., :rot // 2].copy(), y[..., rot // 2:rot].copy()
        y[..., :rot // 2], y[..., rot // 2:rot] = bf16(a * cos - b * sin), bf16(b * cos + a * sin)
    return y


def attention(q, kvals, vvals, kscales, vscales, table, lens, page, causal, scale, q_lens=None):
    """q [B, H_q, S_q, D]; returns o, lse and the bounds of their errors (NaN-free inputs)."""
    B, Hq, Sq, D = q.shape
    H = kvals.shape[1]
    R = Hq // H
    o = np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    o_tol, lse_tol = np.zeros(q.shape), np.zeros(q.shape[:3])
    four = kscales is not None
    for b in range(B):
        L = int(lens[b])
        nq = Sq if q_lens is None else int(q_lens[b])
        if L == 0:
            continue
        k, v = gather(kvals, table[b], L, page), gather(vvals, table[b], L, page)
        if four:
            vs = gather(vscales, table[b], L, page)
        for h in range(Hq):
            kh, vh = k[h // R], v[h // R]
            for i in range(nq):
                n = max(0, min(L, L - nq + i + 1)) if causal else L
                if n == 0:
                    continue
                x = q[b, h, i]
                s = scale * (kh[:n] @ x)
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                o[b, h, i] = p @ vh[:n] / l
                lse[b, h, i] = m + np.log(l)
                A = p @ np.abs(vh[:n]) / l
                es = abs(scale) * (np.abs(kh[:n]) @ np.abs(x)) * 2.0 ** -18
                if four:
                    es = es + abs(scale) * np.abs(kh[:n]).sum(-1) * np.abs(x).max() * 2.0 ** -25
                e = float(es.max()) + np.abs(s).max() * 1.5 * 2.0 ** -22 + 2.0 ** -22
                share = 2.0 ** -11 if four else 2.0 ** -8
                tol = (1.01 * (share + 2 * e)) * A
                if four:
                    tol = tol + n * 2.0 ** -27 * vs[h // R][:n].max()
                o_tol[b, h, i] = tol + 2.0 ** -8 * (np.abs(o[b, h, i]) + tol) + 1e-37
                lse_tol[b, h, i] = e + 2.0 ** -20 * (1 + abs(lse[b, h, i]))
    return o, lse, o_tol, lse_tol
