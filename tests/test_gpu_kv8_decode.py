"""gdn_attn_decode_kv8 against the 64-bit form (tests/_kv8.py has the bound): lengths of 0
and 1 and around pages, blocks, units and runs, every head dim, type, page size and
group size, blocks of very different scales, scores that grow, collected weights,
what lies beyond a sequence, bad pages and lengths, strides, streams and graphs."""
import math

import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _attn, _kv8
from tests._attn import IO, normal

pytestmark = pytest.mark.gpu


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _workspace(dims, n, capacity=0):
    # whatever an earlier call left there must not matter: NaN bytes
    size = gdn.gdn_attn_decode_kv8_workspace_size(dims, n, capacity)
    return torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")


def _on_gpu(cache):
    return gdn.Kv8Cache(*(t.cuda() for t in cache))


CASES = [   # lengths, hq, hkv, d, page, io, gate
    ([1], 2, 1, 64, 16, "bf16", False),
    ([1], 16, 4, 256, 64, "bf16", True),
    ([700], 16, 4, 256, 64, "bf16", True),
    ([5000], 4, 2, 128, 128, "fp16", False),
    ([0, 1, 0, 15, 16, 17, 0], 4, 2, 256, 64, "bf16", True),
    ([127, 128, 129, 257, 2], 6, 2, 64, 16, "fp16", True),
    ([31, 32, 500], 3, 3, 256, 32, "fp16", False),
    ([100, 7], 40, 2, 128, 64, "bf16", True),           # groups of twenty: two items
    ([200, 90], 16, 1, 256, 16, "bf16", False),         # sixteen heads
    ([300, 1], 12, 1, 64, 32, "fp16", True),
    ([130, 260], 9, 1, 256, 128, "bf16", False),
    (list(range(1, 400, 9)), 4, 2, 64, 32, "bf16", False),
    ([0, 0, 0], 4, 2, 128, 32, "bf16", True),
    ([3] * 400, 2, 1, 64, 16, "bf16", False),           # more rows than a CTA has threads
    ([1500, 40, 900], 48, 2, 64, 64, "bf16", True),     # groups of 24
    ([2000, 1100], 8, 8, 128, 64, "fp16", False),
    ([30_001, 3], 4, 1, 256, 128, "bf16", False),
    # many short rows beside a long one: a merge by borders, an item of nearly all runs
    ([5] * 400 + [9000, 0, 300] + [7] * 300, 16, 1, 64, 16, "bf16", False),
    ([1, 0, 70] * 120 + [2500], 4, 2, 128, 64, "fp16", True),
]


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("lens,hq,hkv,d,page,io,gate", CASES)
def test_decode(gpu_lib, lens, hq, hkv, d, page, io, gate, weights):
    g = torch.Generator().manual_seed(sum(lens) + d)
    dt, n = IO[io], len(lens)
    cache = _kv8.paged(g, lens, hkv, d, page)
    qg = normal(g, n, hq, 2 * d, dtype=dt)
    dims = gdn.make_attn_dims(hq, hkv, d, io=io, page_size=page)
    qgd, status = qg.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    ref, slack, w, ws = _kv8.decode(qg[..., :d], cache, lens, qg[..., d:] if gate else None,
                                    _attn.scale_of(d), dt)
    # a table that could hold long sequences, its other entries no pages at all: the form for
    # few keys does not apply
    table = cache[4]
    wide = torch.full((n, max(table.shape[1], 16384 // page)), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    for what, tb in (("few", table), ("wide table", wide)):
        c = _on_gpu((*cache[:4], tb))
        cap = tb.shape[1] * page
        old = torch.rand(n, hkv, cap, generator=g) if weights else None
        got = old.cuda() if weights else None
        o = gdn.gdn_attn_decode_kv8(dims, qgd[..., :d], c, _ints(lens),
                                    _workspace(dims, n, cap if weights else 0),
                                    gate=qgd[..., d:] if gate else None, weights=got, d_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        _attn.check(o, ref, slack, dt, what)
        if weights:
            _kv8.check_weights(got, old, w, ws, what)


@pytest.mark.parametrize("hq,hkv,d,page,io", [(8, 2, 256, 64, "bf16"), (12, 1, 256, 16, "fp16"),
                                               (8, 2, 128, 128, "fp16"), (32, 2, 128, 32, "bf16"),
                                               (4, 4, 64, 64, "bf16"), (10, 1, 64, 16, "bf16")])
def test_runs_that_go_round_the_stages_many_times(gpu_lib, hq, hkv, d, page, io):
    """The same keys again and again (pages that a block table names many times) leave the softmax's
    average as it is: the reference is one cycle."""
    g = torch.Generator().manual_seed(d + hq)
    n, cycle, times = 9, 1024, 128
    dt = IO[io]
    cache = _kv8.paged(g, [cycle] * n, hkv, d, page)
    table = cache[4].repeat(1, times)
    q = normal(g, n, hq, d, dtype=dt)
    ref, slack, w, ws = _kv8.decode(q, cache, [cycle] * n, None, _attn.scale_of(d), dt)
    # the sums are of `times` as many terms
    slack += cycle * times * 2.0 ** -24 * ref.abs().max() * 4
    dims = gdn.make_attn_dims(hq, hkv, d, io=io, page_size=page)
    c, cap = _on_gpu((*cache[:4], table)), cycle * times
    status, got = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(n, hkv, cap, device="cuda")
    for lens in ([cap] * n, [cap - 1, 1, 5] * 3):
        got.zero_()
        o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), c, _ints(lens), _workspace(dims, n, cap),
                                    weights=got, d_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        if lens[1] == cap:
            _attn.check(o, ref, slack, dt, "o")
            for t in (0, 1, times // 2, times - 1):
                part = got[..., t * cycle:(t + 1) * cycle].double().cpu()
                off = (part - w / times).abs() - ws / times - cycle * times * 2.0 ** -24 * part
                assert (off <= 2.0 ** -116).all(), float(off.max())


def _rescaled(cache, lens, page, exps, which):
    """The cache with the scales of each sequence's blocks set to 2^exps, in turn."""
    cache = tuple(t.clone() for t in cache)
    for b, length in enumerate(lens):
        for blk in range(-(-length // 16)):
            pg, i = int(cache[4][b, blk * 16 // page]), blk * 16 % page // 16
            cache[2 + which][pg, :, i] = 2.0 ** exps[blk % len(exps)]
    return cache


@pytest.mark.parametrize("exps", [[-40, 40], [40, -40], [0, -40, 12, -12], [-40], [40],
                                  list(range(-40, 41, 5)), list(range(40, -41, -5))])
@pytest.mark.parametrize("d,page", [(64, 16), (256, 64)])
def test_values_of_very_different_scales(gpu_lib, exps, d, page):
    g = torch.Generator().manual_seed(len(exps) + d)
    lens, hq, hkv = [300, 40, 17], 4, 2
    cache = _rescaled(_kv8.paged(g, lens, hkv, d, page), lens, page, exps, 1)
    q = normal(g, 3, hq, d)
    dims = gdn.make_attn_dims(hq, hkv, d, page_size=page)
    ref, slack, _, _ = _kv8.decode(q, cache, lens, None, _attn.scale_of(d), torch.bfloat16)
    o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), _on_gpu(cache), _ints(lens), _workspace(dims, 3))
    torch.cuda.synchronize()
    _attn.check(o, ref, slack, torch.bfloat16, "o")


def test_a_large_block_that_is_not_attended_to_hides_nothing(gpu_lib):
    """Values of 2^40 with a weight far below 2^-40 beside ordinary ones."""
    d, page, length = 64, 16, 32
    codes = torch.ones(2, 1, page, d)
    k, v = codes.clone(), codes.clone()
    k[0] *= -8      # the first block: scores of -(8 * 8 * 64) / 8 = -512
    k[1] *= 8
    cache = (_kv8.codes_of(k), _kv8.codes_of(v), torch.ones(2, 1, 1), torch.tensor([2.0 ** 40, 1.0]).view(2, 1, 1),
             torch.tensor([[0, 1]], dtype=torch.int32))
    q = torch.full((1, 1, d), 8.0).bfloat16()
    dims = gdn.make_attn_dims(1, 1, d, page_size=page)
    for order in ([0, 1], [1, 0]):
        c = (*cache[:4], torch.tensor([order], dtype=torch.int32))
        o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), _on_gpu(c), _ints([length]), _workspace(dims, 1))
        torch.cuda.synchronize()
        assert (o == 1).all(), order


@pytest.mark.parametrize("exps", [[0, 6, -6], list(range(-8, 9))])
def test_scores_of_very_different_scales(gpu_lib, exps):
    g = torch.Generator().manual_seed(7)
    lens, hq, hkv, d, page = [500, 129], 8, 2, 128, 32
    cache = _rescaled(_kv8.paged(g, lens, hkv, d, page), lens, page, [e - 8 for e in exps], 0)
    q = normal(g, 2, hq, d) * torch.exp2(torch.arange(-20.0, 28.0, 6.0))[None, :, None].bfloat16()
    for scale in (None, 0.02, 1.5):
        dims = gdn.make_attn_dims(hq, hkv, d, page_size=page, scale=scale)
        real = float(torch.tensor(scale or _attn.scale_of(d)))
        ref, slack, w, ws = _kv8.decode(q, cache, lens, None, real, torch.bfloat16)
        c = _on_gpu(cache)
        got = torch.zeros(2, hkv, c.block_table.shape[1] * page, device="cuda")
        o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), c, _ints(lens), _workspace(dims, 2, got.shape[2]),
                                    weights=got)
        torch.cuda.synchronize()
        _attn.check(o, ref, slack, torch.bfloat16, f"scale {scale}")
        _kv8.check_weights(got, torch.zeros_like(got), w, ws, f"scale {scale}")


def test_scales_of_zero(gpu_lib):
    """Blocks whose values, or keys, are all zeros by their scale."""
    g = torch.Generator().manual_seed(3)
    lens, hq, hkv, d, page = [100, 16, 33], 4, 2, 128, 16
    for which in (0, 1):
        cache = tuple(t.clone() for t in _kv8.paged(g, lens, hkv, d, page))
        for b, length in enumerate(lens):
            for blk in range(0, -(-length // 16), 2):
                cache[2 + which][int(cache[4][b, blk])] = 0.0
        q = normal(g, 3, hq, d)
        dims = gdn.make_attn_dims(hq, hkv, d, page_size=page)
        ref, slack, _, _ = _kv8.decode(q, cache, lens, None, _attn.scale_of(d), torch.bfloat16)
        o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), _on_gpu(cache), _ints(lens), _workspace(dims, 3))
        torch.cuda.synchronize()
        _attn.check(o, ref, slack, torch.bfloat16, f"kind {which}")


def test_queries_of_every_size(gpu_lib):
    """Rows of zeros, of the smallest and of the largest numbers, with outliers."""
    g = torch.Generator().manual_seed(9)
    lens, hq, hkv, d, page = [70], 8, 1, 64, 16
    cache = _kv8.paged(g, lens, hkv, d, page)
    q = normal(g, 1, hq, d)
    q[0, 0] = 0
    q[0, 1] *= 2.0 ** -100
    q[0, 2] *= 2.0 ** -125
    q[0, 3, 0] = 2.0 ** 15
    q[0, 4] *= 2.0 ** 10
    q[0, 5, :32] *= 2.0 ** -30
    dims = gdn.make_attn_dims(hq, hkv, d, page_size=page)
    ref, slack, _, _ = _kv8.decode(q, cache, lens, None, _attn.scale_of(d), torch.bfloat16)
    o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), _on_gpu(cache), _ints(lens), _workspace(dims, 1))
    torch.cuda.synchronize()
    _attn.check(o, ref, slack, torch.bfloat16, "o")
    q[0, 6, 3], q[0, 7, 3] = math.nan, math.inf
    o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), _on_gpu(cache), _ints(lens), _workspace(dims, 1))
    torch.cuda.synchronize()
    assert torch.isnan(o[0, 6]).all() and torch.isnan(o[0, 7]).all()
    _attn.check(o[:, :6], ref[:, :6], slack[:, :6], torch.bfloat16, "beside rows that are not finite")


def test_bad_pages_and_lengths(gpu_lib):
    g = torch.Generator().manual_seed(5)
    lens, hq, hkv, d, page = [64, 200, 30], 4, 2, 128, 16
    cache = _kv8.paged(g, lens, hkv, d, page)
    q = normal(g, 3, hq, d)
    dims = gdn.make_attn_dims(hq, hkv, d, page_size=page)
    table = cache[4].clone()
    table[0, 2], table[2, 1] = -7, 1 << 30
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref, slack, _, _ = _kv8.decode(q, cache, lens, None, _attn.scale_of(d), torch.bfloat16)
    o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), _on_gpu((*cache[:4], table)), _ints(lens),
                                _workspace(dims, 3), d_status=status)
    torch.cuda.synchronize()
    assert status.item() == gdn.GDN_DEV_BAD_PAGE
    _attn.check(o[1:2], ref[1:2], slack[1:2], torch.bfloat16, "the row beside")
    # longer than the table holds: cut to it; less than nothing: zeros
    status.zero_()
    full = [table.shape[1] * page] * 3
    cache = _kv8.paged(g, full, hkv, d, page)
    ref, slack, w, ws = _kv8.decode(q, cache, [full[0], full[0], 0], None, _attn.scale_of(d), torch.bfloat16)
    got = torch.zeros(3, hkv, full[0], device="cuda")
    o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), _on_gpu(cache), _ints([full[0], 1 << 30, -3]),
                                _workspace(dims, 3, full[0]), weights=got, d_status=status)
    torch.cuda.synchronize()
    assert status.item() == gdn.GDN_DEV_BAD_LENGTH
    _attn.check(o, ref, slack, torch.bfloat16, "o")
    _kv8.check_weights(got, torch.zeros_like(got), w, ws, "weights")


def test_in_a_graph_on_other_streams_and_the_same_twice(gpu_lib):
    g = torch.Generator().manual_seed(6)
    lens, hq, hkv, d, page = [900, 70, 4000], 8, 2, 256, 64
    c = _on_gpu(_kv8.paged(g, lens, hkv, d, page))
    q, n = normal(g, 3, hq, d).cuda(), _ints(lens)
    dims = gdn.make_attn_dims(hq, hkv, d, page_size=page)
    cap = c.block_table.shape[1] * page
    ws, w = _workspace(dims, 3, cap), torch.zeros(3, hkv, cap, device="cuda")
    o = gdn.gdn_attn_decode_kv8(dims, q, c, n, ws, weights=w)
    torch.cuda.synchronize()
    first = w.clone()
    graph, o2 = torch.cuda.CUDAGraph(), torch.empty_like(o)
    w.zero_()
    with torch.cuda.graph(graph):
        gdn.gdn_attn_decode_kv8(dims, q, c, n, ws, weights=w, o=o2)
    for _ in range(2):
        w.zero_()
        o2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(first, w)
    # other lengths in the same graph
    n.copy_(_ints([1, 0, 130]))
    graph.replay()
    again = gdn.gdn_attn_decode_kv8(dims, q, c, n, _workspace(dims, 3))
    torch.cuda.synchronize()
    assert torch.equal(again, o2)
    # two calls at once, each with its workspace
    n.copy_(_ints(lens))
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    both = [gdn.gdn_attn_decode_kv8(dims, q, c, n, _workspace(dims, 3), stream=s.cuda_stream)
            for s in side]
    torch.cuda.synchronize()
    assert all(torch.equal(o, x) for x in both)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens,hq,hkv,d", [([700], 4, 2, 256), ([200, 900], 4, 2, 128), ([90], 2, 1, 64),
                                           ([400], 16, 1, 256)])
def test_a_wait_that_runs_out_is_reported(gpu_lib, lens, hq, hkv, d, wide):
    """The waits give up after 2 ms here and one CTA goes without a unit of keys: reported, the
    rows that it has no share in right, the next call as if nothing had been."""
    g = torch.Generator().manual_seed(d)
    page = 64
    cache = _kv8.paged(g, lens, hkv, d, page)
    q = normal(g, len(lens), hq, d)
    if wide:
        table = torch.full((len(lens), 256), -1, dtype=torch.int32)
        table[:, :cache[4].shape[1]] = cache[4]
        cache = (*cache[:4], table)
    ref, slack, _, _ = _kv8.decode(q, cache, lens, None, _attn.scale_of(d), torch.bfloat16)
    c = _on_gpu(cache)

    def call(flags):
        dims = gdn.make_attn_dims(hq, hkv, d, page_size=page, flags=flags)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), c, _ints(lens), _workspace(dims, len(lens)),
                                    d_status=status)
        torch.cuda.synchronize()
        return o, status.item()
    o, status = call(gdn.GDN_TEST_WAIT_TIMEOUT)
    assert status == gdn.GDN_DEV_WAIT_TIMEOUT
    rows = torch.isfinite(o).all(-1).cpu()
    assert not rows.all()
    _attn.check(o.cpu()[rows], ref[rows], slack[rows], torch.bfloat16, "the other rows")
    o, status = call(0)
    assert status == 0
    _attn.check(o, ref, slack, torch.bfloat16, "the next call")
