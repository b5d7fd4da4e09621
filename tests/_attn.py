"""Plain 64-bit forms of the full-attention operators and the error bounds
their tests use.

With u the half step of the I/O type (torch.finfo(t).eps / 2) and e = 2^-24:

norm + rotation   everything before the one rounding is fp32: the sum of
  squares (a tree, 13 roundings at most), the root, the weight, the angle's
  cosine and sine (2^-22 absolute) and the two products and their sum come to
  less than 32 e of the pair's |a| + |b|; then u |y|.
attention   a score is a d-term sum of products exact in fp32, accumulated in
  fp32 with truncation at worst: off by 2 d e scale sum |q k|, which is the
  relative error of a weight (twice: numerator and sum).  2^x and the sums add
  less than 64 e + keys e.  Every weight is rounded to the I/O type for the
  product with v (u), so with A = sum p |v| / sum p
    |err| <= u |o| + (u + 4 d e scale max sum |q k| + 64 e + keys e) A,
  and the gate's sigmoid adds 16 e |o|.
"""
import math

import torch

E = 2.0 ** -24
IO = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_step(t):
    return torch.finfo(t).eps / 2


def normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, dtype=torch.float32).to(dtype)


def norm_rope(x, w, eps, pos, freq, layout, rope_scale=1.0):
    """(y, bound without the output rounding) of x [n, h, d] in 64 bits."""
    x = x.double()
    if w is not None:
        x = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    y, size = x.clone(), x.abs()
    half = freq.numel()
    for i in range(half):
        a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
        c = (pos.double() * freq[i]).cos()[:, None] * rope_scale
        s = (pos.double() * freq[i]).sin()[:, None] * rope_scale
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
        size[..., a] = size[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(rope_scale)
    return y, 32 * E * size


def attend(q, k, v, seen, scale):
    """(o, bound's A, score term) of rows q [r, d] over k, v [s, d]; row i sees
    the first seen[i] keys."""
    r, d = q.shape
    o, a = torch.zeros(r, d, dtype=torch.float64), torch.zeros(r, d, dtype=torch.float64)
    es = torch.zeros(r, 1, dtype=torch.float64)
    q, k, v = q.double(), k.double(), v.double()
    for i in range(r):
        n = int(seen[i])
        if n <= 0:
            continue
        s = (k[:n] @ q[i]) * scale
        p = torch.exp(s - s.max())
        p = p / p.sum()
        o[i] = p @ v[:n]
        a[i] = p @ v[:n].abs()
        es[i] = 4 * d * E * scale * (k[:n].abs() @ q[i].abs()).max() + (64 + n) * E
    return o, a, es


def gated(o, gate):
    return o if gate is None else o * torch.sigmoid(gate.double())


def check(got, ref, slack, io, what):
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    # fp16 has a smallest step: half of it, below its normal range
    tiny = 2.0 ** -25 if io == torch.float16 else 0.0
    bound = half_step(io) * ref.abs() + (1 + half_step(io)) * slack + tiny
    over = (got - ref).abs() - bound
    assert (over <= 0).all(), (f"{what}: {int((over > 0).sum())} of {over.numel()} outside the bound,"
                               f" worst by {float(over.max()):.3e}")


def prefill(q, k, v, cu_q, cu_kv, gate, scale, io):
    """(o, slack) of packed causal attention; host lists cu_q, cu_kv."""
    hq, hkv = q.shape[1], k.shape[1]
    o = torch.zeros(q.shape, dtype=torch.float64)
    slack = torch.zeros_like(o)
    u = half_step(io)
    for b in range(len(cu_q) - 1):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_kv[b + 1] - cu_kv[b]
        seen = torch.arange(lq) + 1 + lk - lq
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_kv[b], cu_kv[b + 1])
        for h in range(hq):
            j = h // (hq // hkv)
            o[rows, h], a, es = attend(q[rows, h], k[keys, j], v[keys, j], seen, scale)
            slack[rows, h] = (u + es) * a
    y = gated(o, gate)
    if gate is not None:
        slack = gated(slack, gate) + 16 * E * o.abs()
    return y, slack


def decode(q, kc, vc, table, lens, gate, scale, io):
    """(o, slack) of one-token attention over a paged cache."""
    n, hq, d = q.shape
    hkv, page = kc.shape[1], kc.shape[2]
    o = torch.zeros(q.shape, dtype=torch.float64)
    slack = torch.zeros_like(o)
    u = half_step(io)
    for b in range(n):
        length = max(int(lens[b]), 0)
        pages = table[b, :-(-length // page)].long()
        for j in range(hkv):
            g = hq // hkv
            k = kc[pages, j].reshape(-1, d)[:length]
            v = vc[pages, j].reshape(-1, d)[:length]
            hs = slice(j * g, (j + 1) * g)
            o[b, hs], a, es = attend(q[b, hs], k, v, [length] * g, scale)
            slack[b, hs] = (u + es) * a
    y = gated(o, gate)
    if gate is not None:
        slack = gated(slack, gate) + 16 * E * o.abs()
    return y, slack


def paged(gen, lens, hkv, d, page, dtype, spare=3, shared=0, fill=float("nan")):
    """A cache for sequences of these lengths (the first `shared` tokens common
    to all), pages in random places; every row that no sequence holds is `fill`.
    Returns (k cache, v cache, block table)."""
    sp = shared // page
    own = [max(-(-v // page) - sp, 0) for v in lens]
    pool = sp + sum(own) + spare
    ids = torch.randperm(pool, generator=gen).to(torch.int32)
    width = max(1, sp, max([sp + u for u in own], default=1))
    table = torch.full((len(lens), width), pool - 1, dtype=torch.int32)
    table[:, :sp] = ids[:sp]
    at = sp
    kc = torch.full((pool, hkv, page, d), fill, dtype=dtype)
    vc = torch.full((pool, hkv, page, d), fill, dtype=dtype)
    for c in (kc, vc):
        for i in ids[:sp].tolist():
            c[i] = normal(gen, hkv, page, d, dtype=dtype)
    for b, u in enumerate(own):
        table[b, sp:sp + u] = ids[at:at + u]
        for j in range(u):
            rows = min(page, lens[b] - (sp + j) * page)
            for c in (kc, vc):
                c[int(ids[at + j]), :, :rows] = normal(gen, hkv, rows, d, dtype=dtype)
        at += u
    return kc, vc, table


def scale_of(d):
    return 1.0 / math.sqrt(d)
