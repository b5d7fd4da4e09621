"""Blocks whose scale is 0 stand for zeros whatever their codes are: what gdn_kv8_append makes of one
that a sequence goes on in, straight from such a cache and behind an eviction, by either of
its kernels, as gather and decode see it; and blocks that go on under a scale that is none."""
import math

import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _attn, _kv8
from tests._attn import IO, normal

pytestmark = pytest.mark.gpu


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _ends(lens):
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    return cu


def _held(g, dims, starts, width, zero):
    """A cache whose sequences hold `starts` tokens of random codes under scales of 2^-12 to 2^-6 (keys)
    and 2^-6 to 2^6 (values), the block that each goes on in under a scale of 0 for its keys (zero
    has 0), its values (1); and the same per sequence, head and kind as tests/_kv8.py has it."""
    page, h, d, n = dims.page_size, dims.h_kv, dims.d, len(starts)
    table = torch.randperm(n * width + 2, generator=g)[:n * width].to(torch.int32).view(n, width)
    c = gdn.make_kv8_cache(dims, n * width + 2, table.cuda())
    for x in c[:2]:
        codes = torch.randint(1, 0x7f, x.shape, generator=g, dtype=torch.uint8)
        codes += 0x80 * torch.randint(0, 2, x.shape, generator=g, dtype=torch.uint8)
        x.view(torch.uint8).copy_(codes)
    for kind, s in enumerate(c[2:4]):
        low, high = ((-12, -5), (-6, 7))[kind]
        s.copy_(torch.exp2(torch.randint(low, high, s.shape, generator=g).float()))
        for b, start in enumerate(starts):
            if kind in zero and start % 16:
                s[int(table[b, start // page]), :, start % page // 16] = 0.0
    want = [[[_kv8.Sequence(d) for _ in range(h)] for _ in range(2)] for _ in range(n)]
    for kind in (0, 1):
        codes, scales = c[kind].view(torch.uint8).cpu().view(_kv8.F8).double(), c[2 + kind].cpu()
        for b, start in enumerate(starts):
            for j in range(h):
                seq = want[b][kind][j]
                seq.codes = codes[table[b].long(), j].reshape(-1, d)[:start].clone()
                seq.scales = scales[table[b].long(), j].reshape(-1)[:-(-start // 16)].tolist()
    return c, want


def _check(dims, cache, want, lens, io):
    """Values as decode and gather take them; the scales of what a block holds."""
    k, v = gdn.gdn_kv8_gather(dims, cache, _ints(_ends(lens)), sum(lens))
    torch.cuda.synchronize()
    at, page = 0, dims.page_size
    table, scales = cache.block_table.cpu(), [x.cpu() for x in cache[2:4]]
    for b, length in enumerate(lens):
        for j in range(dims.h_kv):
            for kind, got in ((0, k), (1, v)):
                seq = want[b][kind][j]
                assert len(seq.codes) == length
                assert torch.equal(got[at:at + length, j].cpu().double(),
                                   seq.values().to(io).double()), (b, j, kind)
                s = scales[kind][table[b].long(), j].reshape(-1)[:len(seq.scales)]
                assert s.tolist() == seq.scales, (b, j, kind)
        at += length


def _attention(g, dims, cache, lens, io):
    n, hq, d = len(lens), dims.h_q, dims.d
    q = normal(g, n, hq, d, dtype=io)
    host = tuple(x.cpu() for x in cache)
    ref, slack, _, _ = _kv8.decode(q, host, lens, None, _attn.scale_of(d), io)
    ws = torch.empty(gdn.gdn_attn_decode_kv8_workspace_size(dims, n), dtype=torch.uint8, device="cuda")
    o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), cache, _ints(lens), ws)
    torch.cuda.synchronize()
    _attn.check(o, ref, slack, io, "decode")


# tokens held, tokens appended: one each (no ends), a few, and whole blocks enough for the ring of tiles
CALLS = [([5, 31, 16, 1], None), ([5, 31, 16, 47], [3, 40, 9, 1]), ([9, 20, 3], [2700, 30, 1])]


@pytest.mark.parametrize("zero", [(0,), (1,), (0, 1)])
@pytest.mark.parametrize("d,page,io", [(64, 16, "bf16"), (128, 64, "fp16"), (256, 32, "bf16")])
@pytest.mark.parametrize("starts,rows", CALLS)
def test_append_behind_a_scale_of_zero(gpu_lib, starts, rows, d, page, io, zero):
    g = torch.Generator().manual_seed(d + len(zero) + sum(starts))
    dt, h = IO[io], 2
    dims = gdn.make_attn_dims(2 * h, h, d, io=io, page_size=page)
    lens = [a + b for a, b in zip(starts, rows or [1] * len(starts))]
    cache, want = _held(g, dims, starts, -(-max(lens) // page), zero)
    cu = _ends(rows or [1] * len(starts))
    kv = normal(g, cu[-1], 2 * h, d, dtype=dt)
    kvd = kv.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(cu[-1], dtype=torch.int32, device="cuda")
    gdn.gdn_kv8_append(dims, None, kvd[:, :h], kvd[:, h:], None, None, None, pos, cache, _ints(starts),
                       cu_seqlens=_ints(cu) if rows else None, d_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for b in range(len(starts)):
        for kind in (0, 1):
            for j in range(h):
                want[b][kind][j].append(kv[cu[b]:cu[b + 1], kind * h + j])
    _check(dims, cache, want, lens, dt)
    if max(lens) < 200:
        _attention(g, dims, cache, lens, dt)


def test_append_of_zeros_behind_a_scale_of_zero(gpu_lib):
    g = torch.Generator().manual_seed(1)
    dims = gdn.make_attn_dims(2, 2, 64, page_size=16)
    cache, want = _held(g, dims, [7], 2, (0, 1))
    x, pos = torch.zeros(2, 2, 64).bfloat16(), _ints([0, 0])
    gdn.gdn_kv8_append(dims, None, x.cuda(), x.cuda(), None, None, None, pos, cache, _ints([7]),
                       cu_seqlens=_ints([0, 2]))
    torch.cuda.synchronize()
    for kind in (0, 1):
        for j in range(2):
            want[0][kind][j].append(x[:, j])
            assert want[0][kind][j].scales == [2.0 ** -40] and not want[0][kind][j].codes.any()
    _check(dims, cache, want, [9], torch.bfloat16)


@pytest.mark.parametrize("d,page", [(64, 32), (256, 64)])
def test_append_behind_an_eviction_of_scales_of_zero(gpu_lib, d, page):
    """All that an eviction brings into the last block stood for 0: the block has a scale of 0."""
    g = torch.Generator().manual_seed(d)
    dims, starts, keep = gdn.make_attn_dims(2, 2, d, page_size=page), [90, 75], 40
    cache, _ = _held(g, dims, starts, 3, ())
    table = cache.block_table.cpu()
    for s in cache[2:4]:
        for b in range(2):
            for blk in range(2, 6):                 # places 32 on: the last eight kept are of them
                s[int(table[b, blk * 16 // page]), :, blk * 16 % page // 16] = 0.0
    to = gdn.make_kv8_cache(dims, 6, torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3))
    w = torch.zeros(2, 2, 3 * page, device="cuda")
    lens, kept = gdn.gdn_kv8_evict(dims, cache, w, _ints(starts), keep, to, first=32, last=8)
    torch.cuda.synchronize()
    assert lens.tolist() == [keep, keep] and (kept[..., :32] == torch.arange(32, device="cuda")).all()
    before = [[[None] * 2 for _ in range(2)] for _ in range(2)]
    host = [x.cpu() for x in to]
    for b in range(2):
        for kind in (0, 1):
            for j in range(2):
                c, s = _kv8.of_sequence(host[kind], host[2 + kind], host[4][b], keep, j)
                seq = _kv8.Sequence(d)
                seq.codes, seq.scales = c, s[::16].tolist()
                assert seq.scales[2] == 0.0 and not seq.values()[32:].any()
                before[b][kind][j] = seq
    x, pos = normal(g, 5, 4, d), _ints([0] * 5)
    xd = x.cuda()
    gdn.gdn_kv8_append(dims, None, xd[:, :2], xd[:, 2:], None, None, None, pos, to, lens,
                       cu_seqlens=_ints([0, 1, 5]))
    torch.cuda.synchronize()
    for b, rows in ((0, x[:1]), (1, x[1:])):
        for kind in (0, 1):
            for j in range(2):
                before[b][kind][j].append(rows[:, 2 * kind + j])
    _check(dims, to, before, [keep + 1, keep + 4], torch.bfloat16)
    _attention(g, dims, to, [keep + 1, keep + 4], torch.bfloat16)


@pytest.mark.parametrize("held", [math.nan, math.inf, -1.0, 2.0 ** 41, 2.0 ** -41])
def test_a_block_under_no_scale_takes_new_rows_as_if_it_began_with_them(gpu_lib, held):
    g = torch.Generator().manual_seed(2)
    dims = gdn.make_attn_dims(2, 2, 64, page_size=16)
    cache, _ = _held(g, dims, [7], 1, ())
    for s in cache[2:4]:
        s.fill_(held)
    x, pos = normal(g, 3, 2, 64), _ints([0] * 3)
    gdn.gdn_kv8_append(dims, None, x.cuda(), x.cuda(), None, None, None, pos, cache, _ints([7]),
                       cu_seqlens=_ints([0, 3]))
    torch.cuda.synchronize()
    page = int(cache.block_table[0, 0])
    for kind in (0, 1):
        for j in range(2):
            want = _kv8.Sequence(64)
            want.append(x[:, j])
            assert float(cache[2 + kind][page, j, 0]) == want.scales[0]
            got = cache[kind].view(torch.uint8)[page, j, 7:10].cpu().view(_kv8.F8).double()
            assert torch.equal(got, want.codes)


def test_not_a_number_under_a_scale_of_zero_stays_one(gpu_lib):
    """0 times NaN is NaN, in the append and in an eviction beside a scale that is not 0."""
    dims = gdn.make_attn_dims(2, 2, 64, page_size=16)
    cache = gdn.make_kv8_cache(dims, 2, _ints([[0, 1]]))
    for x in cache[:2]:
        x.view(torch.uint8).fill_(0x35)
        x.view(torch.uint8)[0, :, 3, 10] = 0x7f
    for s in cache[2:4]:
        s[1] = 1.0
    to = gdn.make_kv8_cache(dims, 1, _ints([[0]]))
    w = torch.zeros(1, 2, 32, device="cuda")
    gdn.gdn_kv8_evict(dims, cache, w, _ints([32]), 16, to, first=8, last=8)
    x = torch.ones(1, 2, 64).bfloat16().cuda()
    gdn.gdn_kv8_append(dims, None, x, x, None, None, None, _ints([0]), cache, _ints([7]))
    torch.cuda.synchronize()
    for c, held in ((cache, 7), (to, 8)):
        for x in c[:2]:
            rows = x.view(torch.uint8)[0, :, :held].cpu().view(_kv8.F8).double()
            assert torch.isnan(rows[:, 3, 10]).all()
            rows[:, 3, 10] = 0
            assert not rows.any()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("exp", [0, -40, 40])
@pytest.mark.parametrize("ahead", [1.0, 3.5, 5.0, 6.0, 8.0, 10.0])
def test_what_places_of_scale_zero_outweigh(gpu_lib, ahead, exp, wide):
    """Every other block has values of scale 0 and keys whose scores lead by 8 `ahead` (2^11.5 to
    2^115): what the rest contributes is right down to 2^-76 of the largest weight."""
    g = torch.Generator().manual_seed(int(ahead))
    d, page, lens = 64, 16, [64, 16, 41, 32]
    n, width = len(lens), 4
    dims = gdn.make_attn_dims(2, 1, d, page_size=page)
    _, v, ks, vs, _ = _kv8.paged(g, [width * page] * n, 1, d, page, spare=0)
    k, ks = torch.zeros(n * width, 1, page, d), torch.ones_like(ks)
    vs = torch.full_like(vs, 2.0 ** exp)
    leads = torch.tensor([[1, 0, 0, 1], [0, 0, 0, 0], [0, 1, 0, 1], [0, 1, 1, 0]]).flatten() > 0
    k[leads], vs[leads] = ahead, 0.0
    table = torch.arange(n * width, dtype=torch.int32).view(n, width)
    q = torch.ones(n, 2, d).bfloat16()
    host = (_kv8.codes_of(k), v, ks, vs, table)
    ref, slack, w, _ = _kv8.decode(q, host, lens, None, _attn.scale_of(d), torch.bfloat16)
    for b, length in enumerate(lens):
        codes, _ = _kv8.of_sequence(v, vs, table[b, :-(-length // page)], length, 0)
        slack[b] += 2.0 ** -76 * float(w[b].max()) * codes.abs().sum(0)
    if wide:
        table = torch.cat([table, torch.full((n, 1020), -1, dtype=torch.int32)], 1)
    cache = gdn.Kv8Cache(*(x.cuda() for x in (*host[:4], table)))
    ws = torch.empty(gdn.gdn_attn_decode_kv8_workspace_size(dims, n), dtype=torch.uint8, device="cuda")
    o = gdn.gdn_attn_decode_kv8(dims, q.cuda(), cache, _ints(lens), ws)
    torch.cuda.synchronize()
    _attn.check(o, ref, slack, torch.bfloat16, "o")
