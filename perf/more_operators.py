"""Packed sequences: rotation with several axes, attention and its gradients, as training and prompt programs call them.

Three operators of ``attention_pipelining_gb300`` (declared in ``include/attn_packed.h``).  The tokens of all
sequences of a batch lie one after the other, [T, heads, D]; sequence b is tokens cu[b] .. cu[b + 1] - 1.

* ``rope_packed``      rotates queries and keys by positions with one to four axes (time, height, width), or back
                       (the gradient);
* ``attn_fwd_packed``  attention of every sequence over its own keys, grouped heads, causal or not, O and LSE;
* ``attn_bwd_packed``  the gradients of q, k and v for an upstream gradient of O, given O and LSE.

``listed()`` names the measured cases, ``draw(rng)`` gives more of the same ranges, ``prepare`` makes a case's inputs
on the GPU, ``run`` makes one pass: the framework's calls where ``own`` is set, else the same operators from
elementary torch operations.  ``exact`` gives a pass's outputs in 64 bits.

Formulas, per sequence with n queries and m keys, query head h over key head g = h / (H_q / H_kv):
query i sees key j where j <= i + m - n (causal: the queries are the newest tokens) or always;
s_ij = scale q_i . k_j, LSE_i = ln sum_seen exp(s_ij), O_i = sum_seen exp(s_ij - LSE_i) v_j (no key seen: O_i = 0,
LSE_i = -inf); P_ij = exp(s_ij - LSE_i), dS_ij = P_ij (dO_i . v_j - dO_i . O_i), dv_j = sum P_ij dO_i,
dk_j = scale sum dS_ij q_i (both over the group's heads too), dq_i = scale sum dS_ij k_j.  Rows behind the last
sequence stay as they were.  A pair (a, b) of elements at angle (cos, sin) becomes (a cos - b sin, b cos + a sin),
backwards (a cos + b sin, b cos - a sin); pair d of the rot / 2 pairs, elements d and d + rot / 2 or (interleaved) 2 d
and 2 d + 1, takes row positions[axis][t], column d of the tables, its axis by the sections that the pairs fall into.
"""
import random

import torch

own = False


# ---------------------------------------------------------------- cases


def _attn(name, op, **kw):
    c = dict(name=name, op=op, B=1, H_q=32, H_kv=8, D=128, lo=1, hi=1, keys="same", klo=0, khi=0, causal=True, pad=0,
             det=False, seed=1)
    c.update(kw)
    return c


def _rope(name, **kw):
    c = dict(name=name, op="rope", T=1, H_q=32, H_kv=8, D=128, s0=64, s1=0, s2=0, s3=0, interleaved=False,
             inverse=False, rows=4096, seed=1)
    c.update(kw)
    return c


def listed():
    return [
        # one short prompt: the call's latency is what counts
        _attn("fwd_one_prompt_100", "fwd", lo=100, hi=100),
        # a batch of prompts of very different lengths, the tensors a little longer than their tokens
        _attn("fwd_b16_ragged", "fwd", B=16, lo=37, hi=4001, pad=21, seed=2),
        # one long document
        _attn("fwd_one_16384", "fwd", lo=16384, hi=16384),
        # image encoder: patches see each other within an image, as many key heads as query heads, heads of 64
        _attn("fwd_b24_images_mha_d64", "fwd", B=24, H_q=16, H_kv=16, D=64, lo=64, hi=2304, causal=False, seed=3),
        # pieces of prompts behind cached prefixes, read back as contiguous keys
        _attn("fwd_b8_behind_prefix", "fwd", B=8, lo=1, hi=512, keys="prefix", klo=100, khi=6000, seed=4),
        # gradients of a small batch of short texts, heads of 64
        _attn("bwd_b4_short_d64", "bwd", B=4, H_q=8, H_kv=2, D=64, lo=30, hi=300, seed=5),
        # a training batch: documents of different lengths packed to 12 thousand tokens or so
        _attn("bwd_b12_packed", "bwd", B=12, lo=100, hi=4096, pad=5, seed=6),
        # one long document
        _attn("bwd_one_16384", "bwd", lo=16384, hi=16384),
        # text over images (cross attention: other lengths of keys than of queries), bit-reproducible gradients
        _attn("bwd_b16_cross_mha_d64", "bwd", B=16, H_q=16, H_kv=16, D=64, lo=20, hi=1000, keys="cross", klo=64, khi=2304,
              causal=False, det=True, seed=7),
        # a decoding step's tokens, three axes
        _rope("rope_t32", T=32, s0=16, s1=24, s2=24),
        # a long video with its text: time, height, width
        _rope("rope_video_16384", T=16384, s0=16, s1=24, s2=24, rows=16384, seed=2),
        # the gradient's way back: heads of 64, adjacent pairs, height and width, odd sizes
        _rope("rope_images_back_d64", T=9001, H_q=16, H_kv=16, D=64, s0=13, s1=19, interleaved=True, inverse=True,
              rows=512, seed=3),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm uniform."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "rope"])
    D = rng.choice([64, 128])
    H_kv = rng.choice([1, 2, 4, 8, 16])
    H_q = min(64, H_kv * rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16]))
    H_q -= H_q % H_kv
    seed = rng.randrange(1 << 20)
    if op == "rope":
        T = _log(rng, 1, min(32768, 16384 * 40 // (H_q + H_kv)))
        pairs = rng.choice([D // 2, D // 2, D // 4])
        cuts = sorted(rng.randint(1, pairs) for _ in range(rng.choice([0, 1, 2, 2, 3])))
        s = [b - a for a, b in zip([0] + cuts, cuts + [pairs])] + [0, 0, 0]
        return dict(op=op, T=T, H_q=H_q, H_kv=H_kv, D=D, s0=s[0], s1=s[1], s2=s[2], s3=s[3],
                    interleaved=rng.random() < 0.3, inverse=rng.random() < 0.5, rows=_log(rng, 16, 32768), seed=seed)
    B = _log(rng, 1, 64)
    keys = rng.choice(["same", "same", "same", "prefix", "cross"])
    # at most the products of the listed 16384 tokens, as a padded batch
    most = 16384 * 16384 * 32 // (B * H_q)
    hi = _log(rng, 1, min(16384, 32768 // B, int(most ** 0.5)))
    lo = rng.choice([0, 1, (hi + 1) // 2, hi])
    khi = _log(rng, 1, max(1, min(16384, 65536 // B, most // hi - hi))) if keys != "same" else 0
    return dict(op=op, B=B, H_q=H_q, H_kv=H_kv, D=D, lo=lo, hi=hi, keys=keys,
                klo=rng.choice([0, 1, khi]) if khi else 0, khi=khi, causal=rng.random() < 0.7,
                pad=rng.choice([0, 0, 1, 130]), det=op == "bwd" and rng.random() < 0.4, seed=seed)


def _spread(rng, B, lo, hi):
    """B whole numbers uniform in logarithm over [lo, hi], the last one hi, the first lo."""
    n = [_log(rng, max(lo, 1), max(hi, 1)) if hi else 0 for _ in range(B)]
    n[0] = lo
    n[-1] = hi
    return n


def _lens(case):
    """Every sequence's queries and keys."""
    rng = random.Random(case["seed"])
    n = _spread(rng, case["B"], case["lo"], case["hi"])
    if case["keys"] == "same":
        return n, n
    m = _spread(rng, case["B"], case["klo"], case["khi"])
    rng.shuffle(m)
    return n, [a + b for a, b in zip(n, m)] if case["keys"] == "prefix" else m


def _pairs(case):
    """Pairs of a query and a key that it sees, of one head."""
    total = 0
    for n, m in zip(*_lens(case)):
        if not case["causal"]:
            total += n * m
        else:  # query i of those that see a key sees m - n + i + 1 of them
            first = max(0, n - m)
            total += (m - n + first + 1 + m) * (n - first) // 2
    return total


def work(case):
    D = case["D"]
    if case["op"] == "rope":
        heads, pairs = case["H_q"] + case["H_kv"], case["s0"] + case["s1"] + case["s2"] + case["s3"]
        axes = sum(case[s] > 0 for s in ("s0", "s1", "s2", "s3"))
        return {"bytes": case["T"] * (heads * 4 * D + axes * 4), "flops": case["T"] * heads * pairs * 6}
    n, m = (sum(x) for x in _lens(case))
    rows, cells = n * case["H_q"], m * case["H_kv"]
    if case["op"] == "fwd":
        return {"bytes": rows * (4 * D + 4) + cells * 4 * D, "flops": 4 * D * case["H_q"] * _pairs(case)}
    return {"bytes": rows * (8 * D + 4) + cells * 8 * D, "flops": 10 * D * case["H_q"] * _pairs(case)}


# ---------------------------------------------------------------- inputs


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _ends(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _sections(case):
    return [case[s] for s in ("s0", "s1", "s2", "s3") if case[s] > 0]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    D, H_q, H_kv = case["D"], case["H_q"], case["H_kv"]
    st = dict(case=case)
    if case["op"] == "rope":
        T, sections = case["T"], _sections(case)
        pairs = sum(sections)
        # queries and keys as views of one projection's output [T, (H_q + 2 H_kv) D]
        x = _randn(gen, T, H_q + 2 * H_kv, D).to(torch.bfloat16)
        st["q"], st["k"] = x[:, :H_q], x[:, H_q:H_q + H_kv]
        st["sections"] = sections
        st["positions"] = torch.randint(0, case["rows"], (len(sections), T), generator=gen, device="cuda",
                                        dtype=torch.int32)
        inv = 10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)
        ang = torch.arange(case["rows"], device="cuda", dtype=torch.float64)[:, None] * inv
        st["cos"], st["sin"] = torch.cos(ang).float(), torch.sin(ang).float()
        st["out"] = (torch.zeros(T, H_q, D, dtype=torch.bfloat16, device="cuda"),
                     torch.zeros(T, H_kv, D, dtype=torch.bfloat16, device="cuda"))
        return st
    n, m = _lens(case)
    st["cu_q"] = _ends(n)
    st["cu_k"] = st["cu_q"] if case["keys"] == "same" else _ends(m)
    T_q = max(1, sum(n) + case["pad"])
    T_k = T_q if case["keys"] == "same" else max(1, sum(m) + case["pad"])
    # some channels of the keys larger than others, as projections give them
    big = torch.exp(0.5 * _randn(gen, 1, H_kv, D))
    q, k, v = _randn(gen, T_q, H_q, D), _randn(gen, T_k, H_kv, D) * big, _randn(gen, T_k, H_kv, D)
    if case["keys"] == "same":   # views of one projection's output
        x = torch.cat([q, k, v], 1).to(torch.bfloat16)
        st["q"], st["k"], st["v"] = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
    else:
        x = torch.cat([k, v], 1).to(torch.bfloat16)
        st["q"], st["k"], st["v"] = q.to(torch.bfloat16), x[:, :H_kv], x[:, H_kv:]
    st["scale"] = D ** -0.5
    st["o"] = torch.zeros(T_q, H_q, D, dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.zeros(H_q, T_q, dtype=torch.float32, device="cuda")
    if case["op"] == "bwd":
        _plain_fwd(st)
        st["dout"] = _randn(gen, T_q, H_q, D).to(torch.bfloat16)
        st["grads"] = (torch.zeros(T_q, H_q, D, dtype=torch.bfloat16, device="cuda"),
                       torch.zeros(T_k, H_kv, D, dtype=torch.bfloat16, device="cuda"),
                       torch.zeros(T_k, H_kv, D, dtype=torch.bfloat16, device="cuda"))
    return st


# ---------------------------------------------------------------- one pass


def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _own_fwd(st):
    import attention_pipelining_gb300 as ap
    c = st["case"]
    o, lse = ap.attn_fwd_packed(st["q"], st["k"], st["v"], st["cu_q"], c["causal"], st["scale"],
                                cu_k=None if c["keys"] == "same" else st["cu_k"], out=(st["o"], st["lse"]))
    return {"o": o, "lse": lse}


def _own_bwd(st):
    import attention_pipelining_gb300 as ap
    c = st["case"]
    dq, dk, dv = ap.attn_bwd_packed(st["q"], st["k"], st["v"], st["o"], st["lse"], st["dout"], st["cu_q"], c["causal"],
                                    st["scale"], cu_k=None if c["keys"] == "same" else st["cu_k"], out=st["grads"],
                                    deterministic=c["det"])
    return {"dq": dq, "dk": dk, "dv": dv}


def _own_rope(st):
    import attention_pipelining_gb300 as ap
    c = st["case"]
    q, k = ap.rope_packed(st["q"], st["k"], st["positions"], st["cos"], st["sin"], st["sections"],
                          interleaved=c["interleaved"], inverse=c["inverse"], out=st["out"])
    return {"q": q, "k": k}


_OWN = {"fwd": _own_fwd, "bwd": _own_bwd, "rope": _own_rope}


# ---------------------------------------------------------------- plain forms


def _rows(cu, most):
    """Tokens of a padded batch [B, most], and which of them there are."""
    i = torch.arange(most, device="cuda")
    live = i < (cu[1:] - cu[:-1])[:, None]
    return torch.where(live, cu[:-1, None] + i, 0).long(), live


def _padded(x, at, heads):
    """x [T, heads * R, D] as fp32 [B, heads, rows * R, D]"""
    x = x[at].float()
    B, n, H, D = x.shape
    return x.view(B, n, heads, H // heads, D).permute(0, 2, 1, 3, 4).reshape(B, heads, n * (H // heads), D)


def _seen(st, n, m):
    """Which keys each row of a padded batch sees: [B, 1, n, 1, m]"""
    i, j = torch.arange(n, device="cuda")[:, None], torch.arange(m, device="cuda")
    lq, lk = (st[c][1:] - st[c][:-1] for c in ("cu_q", "cu_k"))
    lq, lk = lq[:, None, None], lk[:, None, None]
    seen = (i < lq) & (j < lk)
    if st["case"]["causal"]:
        seen = seen & (j <= i + lk - lq)
    return seen[:, None, :, None, :]


def _scores(st):
    """Scores of a padded batch [B, H_kv, n * R, m] with -inf for keys not seen, queries, keys, tokens."""
    c = st["case"]
    n, m = (max(1, max(x)) for x in _lens(c))
    at_q, live_q = _rows(st["cu_q"], n)
    at_k, live_k = _rows(st["cu_k"], m)
    q, k = _padded(st["q"], at_q, c["H_kv"]), _padded(st["k"], at_k, c["H_kv"])
    s = (q @ k.transpose(2, 3)).mul_(st["scale"])
    B, H, _, _ = s.shape
    s.view(B, H, n, -1, m).masked_fill_(~_seen(st, n, m), float("-inf"))
    return s, q, k, (at_q, live_q), (at_k, live_k)


def _unpadded(x, rows, heads):
    """[B, H_kv, n * R, ...] back to the tokens that there are [tokens, heads, ...]"""
    at, live = rows
    B, H = x.shape[:2]
    x = x.view(B, H, at.shape[1], heads // H, *x.shape[3:])
    return x.permute(0, 2, 1, 3, *range(4, x.dim())).flatten(2, 3)[live]


def _plain_fwd(st):
    c = st["case"]
    s, q, k, rq, rk = _scores(st)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    v = _padded(st["v"], rk[0], c["H_kv"])
    o = p @ v
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + torch.log(l))[..., 0]
    tokens = rq[0][rq[1]]
    st["o"][tokens] = _unpadded(o, rq, c["H_q"]).to(torch.bfloat16)
    st["lse"][:, tokens] = _unpadded(lse, rq, c["H_q"]).T
    return {"o": st["o"], "lse": st["lse"]}


def _plain_bwd(st):
    c = st["case"]
    s, q, k, rq, rk = _scores(st)
    H = c["H_kv"]
    lse = _padded(st["lse"].T[..., None], rq[0], H)
    lse = torch.where(lse == float("-inf"), torch.zeros_like(lse), lse)
    p = s.sub_(lse).exp_()
    do, o = _padded(st["dout"], rq[0], H), _padded(st["o"], rq[0], H)
    delta = (do * o).sum(-1, keepdim=True)
    v = _padded(st["v"], rk[0], H)
    dv = p.transpose(2, 3) @ do
    ds = (do @ v.transpose(2, 3)).sub_(delta).mul_(p)
    del p, s
    dq = (ds @ k) * st["scale"]
    dk = (ds.transpose(2, 3) @ q) * st["scale"]
    tq, tk = rq[0][rq[1]], rk[0][rk[1]]
    st["grads"][0][tq] = _unpadded(dq, rq, c["H_q"]).to(torch.bfloat16)
    st["grads"][1][tk] = _unpadded(dk, rk, H).to(torch.bfloat16)
    st["grads"][2][tk] = _unpadded(dv, rk, H).to(torch.bfloat16)
    return {"dq": st["grads"][0], "dk": st["grads"][1], "dv": st["grads"][2]}


def _rotated(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    y = x[..., :rot].float()
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:])
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([y.to(torch.bfloat16), x[..., rot:]], -1)


def _plain_rope(st):
    c = st["case"]
    at = torch.cat([p.expand(n, -1) for p, n in zip(st["positions"], st["sections"])]).T.long()   # [T, pairs]
    cos, sin = torch.gather(st["cos"], 0, at)[:, None], torch.gather(st["sin"], 0, at)[:, None]
    sin = -sin if c["inverse"] else sin
    st["out"][0].copy_(_rotated(st["q"], cos, sin, c["interleaved"]))
    st["out"][1].copy_(_rotated(st["k"], cos, sin, c["interleaved"]))
    return {"q": st["out"][0], "k": st["out"][1]}


_PLAIN = {"fwd": _plain_fwd, "bwd": _plain_bwd, "rope": _plain_rope}


# ---------------------------------------------------------------- in 64 bits


def _turn64(x, case, st):
    """Pair by pair from the definition, each pair's axis found by counting through the sections."""
    y = x.double().clone()
    pairs = sum(st["sections"])
    for d in range(pairs):
        axis = 0
        while d >= sum(st["sections"][:axis + 1]):
            axis += 1
        pos = st["positions"][axis].long()
        c, s = st["cos"][pos, d].double()[:, None], st["sin"][pos, d].double()[:, None]
        if case["inverse"]:
            s = -s
        u, w = (2 * d, 2 * d + 1) if case["interleaved"] else (d, d + pairs)
        a, b = x[..., u].double(), x[..., w].double()
        y[..., u], y[..., w] = a * c - b * s, b * c + a * s
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return {"q": _turn64(st["q"], case, st), "k": _turn64(st["k"], case, st)}
    R = case["H_q"] // case["H_kv"]
    q, k, v = (st[x].double().transpose(0, 1) for x in "qkv")                 # [heads, T, D]
    fwd = case["op"] == "fwd"
    if fwd:
        o, lse = torch.zeros_like(q), torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    else:
        do, lse = st["dout"].double().transpose(0, 1), st["lse"].double()
        delta = (do * st["o"].double().transpose(0, 1)).sum(-1)
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    a = b = 0
    for n, m in zip(*_lens(case)):
        for first in range(0, n, 1024):
            rows = slice(a + first, a + min(n, first + 1024))
            last = m - n + min(n, first + 1024) if case["causal"] else m      # keys that the last row sees
            if last <= 0:
                if fwd:
                    lse[:, rows] = float("-inf")
                continue
            i, j = torch.arange(rows.start - a, rows.stop - a, device="cuda"), torch.arange(last, device="cuda")
            hidden = (j[None] > i[:, None] + m - n) if case["causal"] else None
            cols = slice(b, b + last)
            for h in range(case["H_q"]):
                kh, vh = k[h // R, cols], v[h // R, cols]
                s = torch.mm(q[h, rows], kh.T) * st["scale"]
                if hidden is not None:
                    s[hidden] = float("-inf")
                if fwd:
                    z = torch.logsumexp(s, 1)
                    lse[h, rows] = z
                    o[h, rows] = torch.mm(torch.exp(s - torch.where(torch.isinf(z), 0.0, z)[:, None]), vh)
                    continue
                z = lse[h, rows]
                p = torch.exp(s - torch.where(torch.isinf(z), 0.0, z)[:, None])
                g = do[h, rows]
                dv[h // R, cols] += torch.mm(p.T, g)
                ds = p * (torch.mm(g, vh.T) - delta[h, rows][:, None])
                dq[h, rows] = torch.mm(ds, kh) * st["scale"]
                dk[h // R, cols] += torch.mm(ds.T, q[h, rows]) * st["scale"]
        a, b = a + n, b + m
    if fwd:
        return {"o": o.transpose(0, 1).contiguous(), "lse": lse}
    return {"dq": dq.transpose(0, 1).contiguous(), "dk": dk.transpose(0, 1).contiguous(),
            "dv": dv.transpose(0, 1).contiguous()}
