"""gdn_attn_decode_kv8 where runs of very many units meet items of a unit or less, every output and
every weight checked.  A sequence's block table names a small pool's pages again and again in a
random order, so that a 64-bit form is a sum over the pool.

uniform   all keys are 0 and a unit's values are one channel's 1, so that an output counts the keys
  of its channel: w = 1 for every key, the sums are of integers below 2^24 and exact in
  fp32 in any order, and what is left is an exponential of an integer, a quotient and a product
  (64 E) and the output's rounding.  A unit left out or taken twice is 1/8 of a channel.
random    the bound of tests/_kv8.py, where the sums' share is of the terms that one accumulator
  receives: no more keys than a run has, the partial results of an item (306 at most) and
  the warps' (8).
"""
import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _attn, _kv8
from tests._attn import E, IO, normal

pytestmark = pytest.mark.gpu
CONFIGS = [(8, 2, 256, 64, "bf16"), (12, 1, 256, 16, "fp16"), (8, 2, 128, 128, "fp16"),
           (32, 2, 128, 32, "bf16"), (4, 4, 64, 64, "bf16"), (10, 1, 64, 16, "bf16")]
CTAS = 304


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _call(dims, q, cache, lens):
    n, cap = len(lens), cache.block_table.shape[1] * dims.page_size
    size = gdn.gdn_attn_decode_kv8_workspace_size(dims, n, cap)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
    got = torch.zeros(n, dims.h_kv, cap, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), cache, _ints(lens), ws, weights=got, d_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    return o, got


def _lengths(cap):
    return [[cap] * 9, [cap - 1, 1, 5] * 3, [cap - 77, 1, 2000, 1, 1, cap // 3, 5, 64, 0]]


@pytest.mark.parametrize("hq,hkv,d,page,io", CONFIGS)
def test_every_unit_counts_once(gpu_lib, hq, hkv, d, page, io):
    g = torch.Generator().manual_seed(d + hq)
    n, cap, dt = 9, 131_072, IO[io]
    span = max(page, 16384 // d)
    per = span // page
    types = torch.randint(0, d, (n, cap // span), generator=g)     # page c: channel c + 7 j of head j is 1
    table = types.to(torch.int32).repeat_interleave(per, 1)
    codes = torch.zeros(d, hkv, page, d)
    for c in range(d):
        for j in range(hkv):
            codes[c, j, :, (c + 7 * j) % d] = 1
    k, ones = torch.zeros_like(codes), torch.ones(d, hkv, page // 16)
    cache = gdn.Kv8Cache(*(t.cuda() for t in (_kv8.codes_of(k), _kv8.codes_of(codes), ones, ones.clone(), table)))
    dims = gdn.make_attn_dims(hq, hkv, d, io=io, page_size=page)
    q = normal(g, n, hq, d, dtype=dt)
    for lens in _lengths(cap):
        o, got = _call(dims, q, cache, lens)
        ref, w = torch.zeros(n, hq, d, dtype=torch.float64), torch.zeros(n, hkv, cap, dtype=torch.float64)
        for b, length in enumerate(lens):
            of = types[b].repeat_interleave(span)[:length]
            for j in range(hkv):
                counts = torch.bincount((of + 7 * j) % d, minlength=d).double()
                ref[b, j * (hq // hkv):(j + 1) * (hq // hkv)] = counts / max(length, 1)
                if length:
                    w[b, j, :length] = hq // hkv / length
        _attn.check(o, ref, 64 * E * ref, dt, f"o of {lens}")
        _kv8.check_weights(got, torch.zeros_like(got), w, 64 * E * w, f"weights of {lens}")


def _reference(q, cache, table, lens, scale):
    """_kv8.decode, the sums over the pool's keys."""
    k8, v8, ks, vs = cache[:4]
    n, hq, d = q.shape
    pool, hkv, page = k8.shape[:3]
    g, cap = hq // hkv, table.shape[1] * page
    run = (sum(lens) // CTAS + 16384 // d * (4 * n // CTAS + 2)) * hkv
    o, slack = (torch.zeros(q.shape, dtype=torch.float64) for _ in range(2))
    w, ws = (torch.zeros(n, hkv, cap, dtype=torch.float64) for _ in range(2))
    every = torch.arange(pool)
    for j in range(hkv):
        kc, kscale = _kv8.of_sequence(k8, ks, every, pool * page, j)
        vc, vscale = _kv8.of_sequence(v8, vs, every, pool * page, j)
        k, v = kc * kscale[:, None], vc * vscale[:, None]
        bad = ~torch.isfinite(k).all(1)                  # the pool's spare pages: no table names them
        for x in (k, v, vc, vscale):
            x[bad] = 0
        for b, length in enumerate(lens):
            if length == 0:
                continue
            at = (table[b].long()[:, None] * page + torch.arange(page)).flatten()[:length]
            seen = torch.bincount(at, minlength=pool * page).double()
            for h in range(j * g, (j + 1) * g):
                x = q[b, h].double()
                s = ((k @ x) * scale)[at]
                p = torch.exp(s - s.max())
                p = p / p.sum()
                es = 4 * d * E * scale * float((k.abs() @ x.abs())[at].max())
                es += (64 + min(length, run + 314)) * E
                es += 2 * scale * d * 2.0 ** -25 * float(x.abs().max() * k.abs().max())
                total = torch.zeros(pool * page, dtype=torch.float64).index_add(0, at, p)
                o[b, h] = total @ v
                low = 2.0 ** -37 * float((p * vscale[at]).max()) * (seen @ vc.abs())
                slack[b, h] = (2.0 ** -11 + es) * (total @ v.abs()) + low
                w[b, j, :length] += p
                ws[b, j, :length] += (es + 64 * E) * p
    return o, slack, w, ws


@pytest.mark.parametrize("hq,hkv,d,page,io", CONFIGS)
def test_long_and_short_items_side_by_side(gpu_lib, hq, hkv, d, page, io):
    g = torch.Generator().manual_seed(d + hq + 1)
    n, cap, dt = 9, 32_768, IO[io]
    cache = _kv8.paged(g, [512] * n, hkv, d, page)
    pages = cache[4].flatten()
    table = pages[torch.randint(0, len(pages), (n, cap // page), generator=g)]
    on_gpu = gdn.Kv8Cache(*(t.cuda() for t in (*cache[:4], table)))
    dims = gdn.make_attn_dims(hq, hkv, d, io=io, page_size=page)
    q = normal(g, n, hq, d, dtype=dt)
    for lens in _lengths(cap)[1:]:
        o, got = _call(dims, q, on_gpu, lens)
        ref, slack, w, ws = _reference(q, cache, table, lens, _attn.scale_of(d))
        _attn.check(o, ref, slack, dt, f"o of {lens}")
        _kv8.check_weights(got, torch.zeros_like(got), w, ws, f"weights of {lens}")


@pytest.mark.parametrize("hq,hkv,d,page", [(8, 2, 256, 64), (32, 2, 128, 32), (8, 8, 64, 16)])
def test_calls_at_once_with_workspaces_of_their_own(gpu_lib, hq, hkv, d, page):
    """Two calls beside each other on two streams, their partial results and scores in workspaces that
    both are there before either starts (runs of units: the block table is wide)."""
    g = torch.Generator().manual_seed(d)
    lens = [900, 70, 4000, 1, 2500]
    n, cap = len(lens), 16_384
    k8, v8, ks, vs, table = _kv8.paged(g, lens, hkv, d, page)
    wide = torch.full((n, cap // page), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    cache = gdn.Kv8Cache(*(t.cuda() for t in (k8, v8, ks, vs, wide)))
    dims = gdn.make_attn_dims(hq, hkv, d, page_size=page)
    q = normal(g, n, hq, d).cuda()
    o, w = _call(dims, q, cache, lens)
    size = gdn.gdn_attn_decode_kv8_workspace_size(dims, n, cap)
    seq_lens = _ints(lens)
    side = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.full((size,), 0xff, dtype=torch.uint8, device="cuda") for _ in side]
    outs = [[(torch.empty_like(o), torch.zeros_like(w)) for _ in range(10)] for _ in side]
    torch.cuda.synchronize()
    for i in range(10):
        for s, ws, out in zip(side, spaces, outs):
            gdn.gdn_attn_decode_kv8(dims, q, cache, seq_lens, ws, weights=out[i][1], o=out[i][0],
                                    stream=s.cuda_stream)
    torch.cuda.synchronize()
    for out in outs:
        for a, b in out:
            assert torch.equal(a, o) and torch.equal(b, w)
