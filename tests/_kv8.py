"""Plain 64-bit forms of the 8-bit cache's operators and the error bounds their
tests use, beside those of tests/_attn.py (E = 2^-24, u the I/O type's half step).

append   what goes in is off by the norm's and rotation's slack (tests/_attn.py); the
  one rounding to e4m3 is off by half a step: 2^-4 of the value, or 2^-10 of the
  block's scale below its normal range.  Values are stored as they come: exact
  codes and scales are expected of them, and of every growth of a scale.
decode   a score is a d-term sum of products of fp16 numbers, exact in fp32,
  accumulated in fp32 with truncation at worst, as in tests/_attn.py; a query
  element below 2^-14 of its row's largest is off by 2^-25 of that in fp16, so
  a score by scale d 2^-25 max|q| max|k| more.  A weight times its block's scale is
  rounded to fp16: 2^-11 of it, or, below fp16's normal range, 2^-25 of
  2^-12 of the largest contribution of the row (2^-37 of it; the reference
  lags by 2^3.9 at most the other way, which only makes that smaller).
weights  each is off by twice the score's error and the roundings of the
  exponential, quotient and sums (64 E), and the sum with what was there by E;
  an exponential below fp32's normal range, 2^-126, is taken as 0, and with a sum of
  2^-3.9 at least (the reference's lag) 64 heads' come to less than 2^-116.
"""
import math

import torch

from tests._attn import E, half_step

F8 = torch.float8_e4m3fn
BLOCK = 16


def quantise(x):
    """x in 64 bits to the nearest e4m3 number, ties to even, 448 at most."""
    size = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(size - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exponent(top):
    """The smallest e of -40 .. 40 with top <= 448 * 2^e."""
    e = -40
    while e < 40 and top > 448 * 2.0 ** e:
        e += 1
    return e


class Sequence:
    """One sequence of one head and kind as the cache should hold it: codes in 64 bits and
    the scale of every block."""

    def __init__(self, d):
        self.codes, self.scales = torch.zeros(0, d, dtype=torch.float64), []

    def append(self, x):
        """x [rows][d] in one call."""
        x = x.double()
        while len(x):
            r = len(self.codes) % BLOCK
            part, x = x[:BLOCK - r], x[BLOCK - r:]
            s = 2.0 ** exponent(float(part.abs().max()))
            if r == 0:
                self.scales.append(s)
            elif s > self.scales[-1]:
                first = len(self.codes) - r
                self.codes[first:] = quantise(self.codes[first:] * (self.scales[-1] / s))
                self.scales[-1] = s
            self.codes = torch.cat([self.codes, quantise(part / self.scales[-1])])

    def values(self):
        per = torch.tensor(self.scales, dtype=torch.float64).repeat_interleave(BLOCK)
        return self.codes * per[:len(self.codes), None]


def codes_of(x):
    """Codes in 64 bits as float8 (they are such numbers)."""
    return x.float().to(F8)


def paged(gen, lens, hkv, d, page, spread=0.5, spare=3):
    """(k, v, k_scale, v_scale, table) of random sequences, pages in random places; every row
    and scale that no sequence holds is NaN.  spread: of the tokens' sizes (log)."""
    used = [-(-max(v, 0) // page) for v in lens]
    pool = sum(used) + spare
    ids = torch.randperm(pool, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(1, *used)), pool - 1, dtype=torch.int32)
    nb = page // BLOCK
    codes = [torch.full((pool, hkv, page, d), 0x7f, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.full((pool, hkv, nb), math.nan) for _ in range(2)]
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at:at + u]
        for j in range(u):
            rows, p = min(page, lens[b] - j * page), int(ids[at + j])
            for c, s in zip(codes, scales):
                x = torch.randn(hkv, page, d, generator=gen, dtype=torch.float64)
                x *= torch.exp(spread * torch.randn(hkv, page, 1, generator=gen, dtype=torch.float64))
                x[:, rows:] = 0
                top = x.abs().view(hkv, nb, -1).amax(-1)
                e = torch.tensor([[exponent(float(t)) for t in row] for row in top])
                sc = torch.exp2(e.double())
                held = -(-rows // BLOCK)
                q = quantise(x / sc.repeat_interleave(BLOCK, 1)[..., None])
                c[p, :, :rows] = codes_of(q)[:, :rows].view(torch.uint8)
                s[p, :, :held] = sc[:, :held].float()
        at += u
    return (*[c.view(F8) for c in codes], *scales, table)


def of_sequence(codes, scales, pages, length, head):
    """Values in 64 bits of the first `length` places: (codes, scale of each row)."""
    d = codes.shape[-1]
    c = codes.view(torch.uint8)[pages.long(), head].reshape(-1, d)[:length].view(F8).double()
    s = scales[pages.long(), head].reshape(-1).double().repeat_interleave(BLOCK)[:length]
    return c, s


def decode(q, cache, lens, gate, scale, io):
    """(o, slack, weights, weights' slack): weights [n][hkv][longest]."""
    k8, v8, ks, vs, table = cache
    n, hq, d = q.shape
    hkv, page = k8.shape[1], k8.shape[2]
    o, slack = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    most = max(max(lens), 1)
    w, ws = torch.zeros(n, hkv, most, dtype=torch.float64), torch.zeros(n, hkv, most, dtype=torch.float64)
    g = hq // hkv
    for b in range(n):
        length = max(int(lens[b]), 0)
        if length == 0:
            continue
        pages = table[b, :-(-length // page)]
        for j in range(hkv):
            kc, kscale = of_sequence(k8, ks, pages, length, j)
            vc, vscale = of_sequence(v8, vs, pages, length, j)
            k, v = kc * kscale[:, None], vc * vscale[:, None]
            for h in range(j * g, (j + 1) * g):
                x = q[b, h].double()
                s = (k @ x) * scale
                p = torch.exp(s - s.max())
                p = p / p.sum()
                es = 4 * d * E * scale * float((k.abs() @ x.abs()).max()) + (64 + length) * E
                es += 2 * scale * d * 2.0 ** -25 * float(x.abs().max() * k.abs().max())
                o[b, h] = p @ v
                a = p @ v.abs()
                low = 2.0 ** -37 * float((p * vscale).max()) * vc.abs().sum(0)
                slack[b, h] = (2.0 ** -11 + es) * a + low
                w[b, j, :length] += p
                ws[b, j, :length] += (es + 64 * E) * p
    y = o if gate is None else o * torch.sigmoid(gate.double())
    if gate is not None:
        slack = slack * torch.sigmoid(gate.double()) + 16 * E * o.abs()
    return y, slack, w, ws


def evicted(weights, length, keep, first, last):
    """Places that are kept of one head."""
    if length <= keep:
        return list(range(length))
    w = [x if x > 0 else 0.0 for x in weights[:length].tolist()]    # NaN: 0
    middle = sorted(range(first, length - last), key=lambda i: (-w[i], i))[:keep - first - last]
    return sorted([*range(first), *middle, *range(length - last, length)])


def check_weights(got, old, w, ws, what):
    """got = old + w within the bound; [n][hkv][capacity] and w's [..][longest]."""
    got, old = got.double().cpu(), old.double().cpu()
    m = w.shape[2]
    total = old[..., :m] + w
    over = (got[..., :m] - total).abs() - ws - 2 * E * total.abs() - 2.0 ** -116
    assert (over <= 0).all(), f"{what}: worst by {float(over.max()):.3e}"
    assert torch.equal(got[..., m:], old[..., m:]), f"{what}: places behind the sequences changed"


def half(io):
    return half_step(io)
