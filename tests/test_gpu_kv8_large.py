"""The 8-bit cache where many rows or long sequences take another kernel or another way through
one: the ring of tiles against the same rows in small calls, bit for bit, with positions of
several axes, and evictions on both sides of what fits shared memory."""
import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _kv8
from tests._attn import IO, normal

pytestmark = pytest.mark.gpu


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hq,hkv,d,rot,page,io", [(4, 2, 256, 256, 16, "bf16"), (7, 1, 128, 64, 64, "fp16"),
                                                  (3, 3, 64, 32, 128, "bf16"), (0, 5, 64, 64, 32, "bf16")])
def test_many_rows_as_in_small_calls(gpu_lib, hq, hkv, d, rot, page, io, layout):
    g = torch.Generator().manual_seed(d + rot)
    dt, lens = IO[io], [2805, 40, 1]
    n, cu = sum(lens), [0, 2805, 2845, 2846]
    dims = gdn.make_attn_dims(max(hq, hkv), hkv, d, io=io, rot_dim=rot, rope=layout, page_size=page)
    hq = dims.h_q if hq else 0
    q = normal(g, n, hq, d, dtype=dt).cuda() if hq else None
    k, v = normal(g, n, hkv, d, dtype=dt).cuda(), normal(g, n, hkv, d, dtype=dt).cuda()
    k[::97] *= 30                                  # scales of many sizes
    pos = torch.randint(0, 100_000, (4, n), generator=g, dtype=torch.int32).cuda()
    axes = gdn.make_rope_axes([i % 4 for i in range(rot // 2)])
    freq = gdn.rope_frequencies(rot, 1e6, device="cuda")[0]
    w = (1 + 0.1 * torch.randn(2, d, generator=g)).cuda()
    width = -(-max(lens) // page)
    table = torch.randperm(3 * width, generator=g).to(torch.int32).view(3, width).cuda()
    whole, parts = (gdn.make_kv8_cache(dims, 3 * width, table) for _ in range(2))
    k_out = torch.empty_like(k)
    o = gdn.gdn_kv8_append(dims, q, k, v, *w, freq, pos, whole, _ints([0, 0, 0]), cu_seqlens=_ints(cu),
                           axes=axes, k_out=k_out)
    q2, k2 = gdn.gdn_qk_norm_rope_axes(dims, q, k, *w, freq, pos, axes)
    assert torch.equal(k_out, k2) and (not hq or torch.equal(o, q2))
    for b in range(3):                             # 160 rows of one sequence at a time
        for r in range(0, lens[b], 160):
            rows = slice(cu[b] + r, min(cu[b] + r + 160, cu[b + 1]))
            m = rows.stop - rows.start
            ends, starts = [0, 0, 0, 0], [0, 0, 0]
            ends[b + 1:] = [m] * (3 - b)
            starts[b] = r
            gdn.gdn_kv8_append(dims, None, k[rows], v[rows], *w, freq, pos[:, rows].contiguous(), parts,
                               _ints(starts), cu_seqlens=_ints(ends), axes=axes)
    ends = _ints(cu)
    for x, y in zip(gdn.gdn_kv8_gather(dims, whole, ends, n), gdn.gdn_kv8_gather(dims, parts, ends, n)):
        assert torch.equal(x, y)
    for x, y in zip(whole[2:4], parts[2:4]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("lens,keep,first,last", [([49152, 49153, 60000], 20000, 7, 333),
                                                  ([49154, 100], 1, 1, 0), ([70000], 69999, 0, 69999)])
@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_eviction_from_long_sequences(gpu_lib, lens, keep, first, last, kind):
    g = torch.Generator().manual_seed(sum(lens))
    n, hkv, d, page = len(lens), 2, 64, 128
    dims = gdn.make_attn_dims(hkv, hkv, d, page_size=page)
    width, small = -(-max(lens) // page), -(-keep // page)
    cache = gdn.make_kv8_cache(dims, n * width, torch.arange(n * width, dtype=torch.int32,
                                                             device="cuda").view(n, width))
    for x in cache[:2]:
        x.view(torch.uint8).copy_(torch.randint(0, 120, x.shape, generator=g, dtype=torch.uint8))
    for x in cache[2:4]:
        x.fill_(0.5)
    to = gdn.make_kv8_cache(dims, n * small, torch.arange(n * small, dtype=torch.int32,
                                                          device="cuda").view(n, small))
    w = torch.rand(n, hkv, width * page, generator=g)
    w = torch.exp(8 * w) if kind == "spread" else torch.floor(4 * w) - 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty(n, hkv, small * page, device="cuda")
    new, kept = gdn.gdn_kv8_evict(dims, cache, w.cuda(), _ints(lens), keep, to, weights_out=out, first=first,
                                  last=last, d_status=status)
    assert status.item() == 0 and new.tolist() == [min(x, keep) for x in lens]
    kept, out = kept.cpu(), out.cpu()
    before, after = ([x.cpu() for x in c[0].view(torch.uint8)] for c in (cache, to))
    for b in range(n):
        for j in range(hkv):
            want = _kv8.evicted(w[b, j], lens[b], keep, first, last)
            assert kept[b, j, :len(want)].tolist() == want and (kept[b, j, len(want):] == -1).all()
            assert torch.equal(out[b, j, :len(want)], w[b, j][want])
            old = torch.cat([before[b * width + i][j] for i in range(width)])
            now = torch.cat([after[b * small + i][j] for i in range(small)])
            assert torch.equal(now[:len(want)], old[want])
