"""Packed attention, its gradients and the rotation with several axes in 64 bits, from the
definitions of include/attn_packed.h, and the bounds of the CUDA kernels' errors: the reference of
tests/test_gpu_packed.py.

Forward, per element (u = 2^-8 bounds the relative error of a rounding to bf16):

* O is divided by the sum of the rounded probabilities that it was made of, so a rounding d_j of
  p_j changes O by d_j p_j (v_j - O) / sum p: at most u sum_j P_ij |v_j - O|.
* A score's error e_j, which its probability takes as a relative error, enters the same way.  The
  tensor core's fp32 sums: at most 2^-20 of the sum of magnitudes a chain of instructions (eight of
  at most four steps of 2^-23 each at D = 128 give 2^-18); the exponent's three fp32 roundings,
  2^-22 of its magnitude, and 2^-22 of ex2 itself.
* fp32 accumulation over the keys: 2^-23 a step of 16 keys, of sum_j P_ij |v_j|.  The running maximum
  may lag by 2^8, which scales sums and their errors alike.
* O's rounding, u |O|.

LSE: max + log2(sum) in fp32.  The sum takes the probabilities' errors and its own roundings (at most
64 additions a block and one a block, of 2^-24 each); log2, the product and the sum 2^-21 (1 + |lse|).

Backward, per element, with the roundings of P and dS (independent, standard deviation at most
u / sqrt(3)): eight standard deviations of the sum, as in bwd_bound.py (o and lse are inputs here,
so D_i has no rounding of O in it), what fp32 costs (each P_ij off by e_ij; dP_ij and D_i by 2^-18 of their sums of
magnitudes; accumulation as above), and u |gradient|.
"""
import math

import torch

U = 2.0 ** -8
K_SIGMA = 8.0


def bounds(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return c


def seen(n, m, causal, device):
    if not causal:
        return torch.ones(n, m, dtype=torch.bool, device=device)
    i, j = torch.arange(n, device=device)[:, None], torch.arange(m, device=device)
    return j <= i + m - n


def _e(q, k, s, scale):
    """Relative error of a probability: [n, m]"""
    mag = abs(scale) * (q.abs() @ k.abs().T)
    big = torch.where(torch.isfinite(s), s, 0.0).abs()
    return mag * 2.0 ** -18 + (big + big.amax(1, keepdim=True)) * 2.0 ** -22 + 2.0 ** -22


def forward(q, k, v, cu_q, cu_k, causal, scale):
    """q [T_q, H_q, D], k and v [T_k, H_kv, D] float64; cu_q and cu_k lists.  Returns o, lse [H_q, T_q]
    and the bounds of their errors; rows of no sequence are NaN."""
    H_q, R = q.shape[1], q.shape[1] // k.shape[1]
    nan = float("nan")
    o, to = torch.full_like(q, nan), torch.full_like(q, nan)
    lse = torch.full((H_q, q.shape[0]), nan, dtype=torch.float64, device=q.device)
    tl = lse.clone()
    for a0, a1, b0, b1 in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        n, m = a1 - a0, b1 - b0
        if n == 0:
            continue
        see = seen(n, m, causal, q.device)
        for h in range(H_q):
            x, y, z = q[a0:a1, h], k[b0:b1, h // R], v[b0:b1, h // R]
            if m == 0:
                o[a0:a1, h], to[a0:a1, h] = 0, 0
                lse[h, a0:a1], tl[h, a0:a1] = -math.inf, 0
                continue
            s = (scale * (x @ y.T)).masked_fill(~see, -math.inf)
            L = torch.logsumexp(s, 1)
            none = torch.isinf(L)
            P = torch.exp(s - torch.where(none, 0.0, L)[:, None])
            O = P @ z
            e = _e(x, y, s, scale)
            # sum_j w_j |v_j - O|, w = P (u + e), a key at a time of blocks of rows
            W = P * (U * 1.01 + 1.01 * e)
            T = torch.stack([(W[i, :, None] * (z - O[i]).abs()).sum(0) for i in range(n)])
            steps = math.ceil(m / 16) + 1
            T = T + steps * 2.0 ** -23 * (P @ z.abs())
            to[a0:a1, h] = torch.where(none[:, None], 0.0, T + U * (O.abs() + T) + 1e-37)
            o[a0:a1, h], lse[h, a0:a1] = O, L
            t = (P * e).amax(1) * 0 + (P * e).sum(1) * 1.01
            t = t + (64 + math.ceil(m / 128)) * 2.0 ** -24 + 2.0 ** -21 * (1 + torch.where(none, 0.0, L).abs())
            tl[h, a0:a1] = torch.where(none, 0.0, t)
    return o, lse, to, tl


def backward(q, k, v, o, lse, do, cu_q, cu_k, causal, scale):
    """Gradients of q, k, v and their allowances: {"dq": (ref, allowance, sd), ...}; rows of no
    sequence are NaN."""
    H_q, R = q.shape[1], q.shape[1] // k.shape[1]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    var = [torch.zeros_like(t) for t in (q, k, v)]    # of the roundings to bf16
    lin = [torch.zeros_like(t) for t in (q, k, v)]    # what fp32 costs
    for a0, a1, b0, b1 in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        n, m = a1 - a0, b1 - b0
        if n == 0 or m == 0:
            continue
        see = seen(n, m, causal, q.device)
        for h in range(H_q):
            g = h // R
            x, y, z, G = q[a0:a1, h], k[b0:b1, g], v[b0:b1, g], do[a0:a1, h]
            s = (scale * (x @ y.T)).masked_fill(~see, -math.inf)
            L = lse[h, a0:a1]
            P = torch.exp(s - torch.where(torch.isinf(L), 0.0, L)[:, None])
            D = (G * o[a0:a1, h]).sum(1, keepdim=True)
            dP = G @ z.T
            dS = P * (dP - D)
            e = _e(x, y, s, scale) + L.nan_to_num(0, 0, 0).abs()[:, None] * 2.0 ** -22
            eS = dS.abs() * e + P * 2.0 ** -18 * (G.abs() @ z.abs().T +
                                                  (G * o[a0:a1, h]).abs().sum(1, keepdim=True)) \
                + dS.abs() * 2.0 ** -23
            dv[b0:b1, g] += P.T @ G
            dk[b0:b1, g] += scale * (dS.T @ x)
            dq[a0:a1, h] = scale * (dS @ y)
            u3 = U * U / 3
            var[0][a0:a1, h] = scale ** 2 * u3 * ((dS * dS) @ (y * y))
            var[1][b0:b1, g] += scale ** 2 * u3 * ((dS * dS).T @ (x * x))
            var[2][b0:b1, g] += u3 * ((P * P).T @ (G * G))
            acc = lambda c: (math.ceil(c / 16) + 1) * 2.0 ** -23  # noqa: E731
            lin[0][a0:a1, h] = abs(scale) * ((eS + dS.abs() * acc(m)) @ y.abs())
            lin[1][b0:b1, g] += abs(scale) * ((eS + dS.abs() * acc(n * R)).T @ x.abs())
            lin[2][b0:b1, g] += (P * (e + acc(n * R))).T @ G.abs()
    out = {}
    for name, ref, w, t, cu in (("dq", dq, var[0], lin[0], cu_q), ("dk", dk, var[1], lin[1], cu_k),
                                ("dv", dv, var[2], lin[2], cu_k)):
        for x in (ref[:cu[0]], ref[cu[-1]:]):
            x.fill_(float("nan"))
        allow = K_SIGMA * w.sqrt() + 1.01 * t
        out[name] = (ref, allow + U * (ref.abs() + allow) + 1e-37, (w + (U * ref) ** 2 / 3).sqrt())
    return out


def round_bf16(x):
    """Nearest values with 8 significant bits, ties to even (float64, bf16's normal range)."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256), e - 8)


def rope(x, positions, cos, sin, sections, interleaved, inverse):
    """x [T, H, D] float64, pair by pair; rounded to bf16."""
    y = x.clone()
    pairs = sum(sections)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for d in range(pairs):
        row = positions[axis[d]].long()
        c, s = cos[row, d].double()[:, None], sin[row, d].double()[:, None]
        s = -s if inverse else s
        i, j = (2 * d, 2 * d + 1) if interleaved else (d, d + pairs)
        y[..., i] = round_bf16(x[..., i] * c - x[..., j] * s)
        y[..., j] = round_bf16(x[..., j] * c + x[..., i] * s)
    return y
