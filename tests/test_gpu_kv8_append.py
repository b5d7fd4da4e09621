"""gdn_kv8_append and gdn_kv8_gather: every row at its place with the right scale, values
bit for bit, scales that grow from call to call, padding, places and pages that
do not exist, what must stay as it was, and packed rows out of the cache."""
import math

import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _attn, _kv8
from tests._attn import IO, normal

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _ends(lens):
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    return cu


def _cache(dims, seqs, width, seed, spare=2):
    """Pages in random places; every code is 0x55 and every scale NaN until written."""
    pool = seqs * width + spare
    ids = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    c = gdn.make_kv8_cache(dims, pool, ids[:seqs * width].view(seqs, width).contiguous().cuda())
    for x in c[:2]:
        x.view(torch.uint8).fill_(0x55)
    for x in c[2:4]:
        x.fill_(math.nan)
    return c


def _row(cache, which, b, head, place):
    """(codes in 64 bits, scale) of one place."""
    page = cache.k.shape[2]
    pg = int(cache.block_table[b, place // page])
    codes, scales = ((cache.k, cache.k_scale), (cache.v, cache.v_scale))[which]
    return (codes.view(torch.uint8)[pg, head, place % page].view(_kv8.F8).double().cpu(),
            float(scales[pg, head, place % page // 16]))


CASES = [   # calls: rows per sequence of each, hq, hkv, d, rot, page, io
    ([[1]], 2, 1, 64, 16, 16, "bf16"),
    ([[16, 5], [3, 11], [1, 1]], 4, 2, 256, 64, 16, "bf16"),
    ([[15, 17, 0, 40], [1, 16, 33, 0], [100, 0, 0, 9]], 4, 1, 128, 128, 64, "fp16"),
    ([[7, 130], [9, 1]], 3, 3, 64, 32, 128, "bf16"),
    ([[300] + [2] * 20, [1] * 21], 2, 2, 256, 0, 32, "fp16"),
    ([[5] * 300], 2, 1, 64, 16, 16, "bf16"),        # more sequences than a CTA has threads
    ([[700], [900]], 16, 4, 256, 64, 64, "bf16"),
    # whole blocks enough for the ring of tiles, odd starts behind an earlier call
    ([[5, 0, 30], [1300, 1111, 202]], 3, 1, 256, 64, 32, "bf16"),
    ([[2500], [7]], 2, 2, 128, 32, 128, "fp16"),
    ([[1400, 9, 1300]], 4, 4, 64, 64, 16, "bf16"),
]


@pytest.mark.parametrize("calls,hq,hkv,d,rot,page,io", CASES)
def test_append_then_gather(gpu_lib, calls, hq, hkv, d, rot, page, io):
    g = torch.Generator().manual_seed(sum(map(sum, calls)) + d)
    dt, seqs = IO[io], len(calls[0])
    total = [sum(c[b] for c in calls) for b in range(seqs)]
    dims = gdn.make_attn_dims(hq, hkv, d, io=io, rot_dim=rot, page_size=page, norm_eps=EPS)
    cache = _cache(dims, seqs, max(1, -(-max(total) // page)), d)
    freq, _ = gdn.rope_frequencies(rot, 1e5) if rot else (torch.zeros(0, dtype=torch.float64), 1.0)
    wq, wk = 1 + 0.1 * torch.randn(d, generator=g), 1 + 0.1 * torch.randn(d, generator=g)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    held = [0] * seqs
    values = [[_kv8.Sequence(d) for _ in range(hkv)] for _ in range(seqs)]
    keys = [[] for _ in range(seqs)]          # (reference, slack) of each row
    for rows in calls:
        n, cu = sum(rows), _ends(rows)
        qg, kv = normal(g, n, hq, 2 * d, dtype=dt), normal(g, n, 2 * hkv, d, dtype=dt)
        # tokens of many sizes, so that scales grow
        kv *= torch.exp2(torch.randint(-6, 7, (n, 2 * hkv, 1), generator=g)).to(dt)
        pos = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32)
        kvd = kv.cuda()
        k_out = torch.empty(n, hkv, d, dtype=dt, device="cuda")
        q = gdn.gdn_kv8_append(dims, qg.cuda()[..., :d], kvd[:, :hkv], kvd[:, hkv:], wq.cuda(), None,
                               freq.cuda() if rot else None, pos.cuda(), cache, _ints(held),
                               cu_seqlens=_ints(cu), k_out=k_out, d_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        qr, qs = _attn.norm_rope(qg[..., :d], wq, EPS, pos, freq, "half")
        kr, kslack = _attn.norm_rope(kv[:, :hkv], None, EPS, pos, freq, "half")
        _attn.check(q, qr, qs, dt, "q")
        _attn.check(k_out, kr, kslack, dt, "k_out")
        for b in range(seqs):
            for j in range(hkv):
                if rows[b]:
                    values[b][j].append(kv[cu[b]:cu[b + 1], hkv + j])
            keys[b] += [(kr[t], kslack[t]) for t in range(cu[b], cu[b + 1])]
            held[b] += rows[b]
    nb = page // 16
    codes_v, scale_v = cache.v.view(torch.uint8).cpu(), cache.v_scale.cpu()
    codes_k, scale_k = cache.k.view(torch.uint8).cpu(), cache.k_scale.cpu()
    seen_rows, seen_blocks = torch.zeros_like(codes_v[..., 0], dtype=torch.bool), torch.zeros_like(scale_v)
    table = cache.block_table.cpu()
    for b in range(seqs):
        for j in range(hkv):
            want = values[b][j]
            for p in range(held[b]):
                pg = int(table[b, p // page])
                seen_rows[pg, j, p % page] = True
                blk = p % page // 16
                seen_blocks[pg, j, blk] = 1
                assert float(scale_v[pg, j, blk]) == want.scales[p // 16]
                got = codes_v[pg, j, p % page].view(_kv8.F8).double()
                assert torch.equal(got, want.codes[p]), (b, j, p)
                # keys: within half a step of their reference (rounded once for every growth)
                ref, slack = keys[b][p][0][j], keys[b][p][1][j]
                s = float(scale_k[pg, j, blk])
                first = p // 16 * 16
                rows16 = keys[b][first:min(first + 16, held[b])]
                top = max(float(r[0][j].abs().max()) for r in rows16)
                off = max(float(r[1][j].max()) for r in rows16)
                assert 2.0 ** _kv8.exponent(top - off) <= s <= 2.0 ** _kv8.exponent(top + off)
                k8 = codes_k[pg, j, p % page].view(_kv8.F8).double() * s
                lost = torch.maximum(ref.abs() * 2.0 ** -4, torch.tensor(s * 2.0 ** -10))
                # an earlier, smaller scale rounded it to no coarser a step; a growth once more
                more = s * 2.0 ** -10 * (len(calls) - 1)
                assert ((k8 - ref).abs() <= lost + more + slack * (1 + 2.0 ** -4)).all(), (b, j, p)
    assert (codes_v[~seen_rows] == 0x55).all() and (codes_k[~seen_rows] == 0x55).all()
    assert torch.isnan(scale_v[seen_blocks == 0]).all() and torch.isnan(scale_k[seen_blocks == 0]).all()
    assert nb * 16 == page
    # out again, packed: what the cache stands for, rounded to the type
    k, v = gdn.gdn_kv8_gather(dims, cache, _ints(_ends(held)), sum(held), d_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    at = 0
    for b in range(seqs):
        for j in range(hkv):
            want = values[b][j].values().to(dt)
            assert torch.equal(v[at:at + held[b], j].cpu(), want)
            c, s = _kv8.of_sequence(cache.k.cpu(), scale_k, table[b, :-(-held[b] // page)], held[b], j)
            assert torch.equal(k[at:at + held[b], j].cpu(), (c * s[:, None]).to(dt))
        at += held[b]


def _one(d=64, hkv=2, page=16, seqs=3, width=2, rot=0):
    dims = gdn.make_attn_dims(hkv, hkv, d, rot_dim=rot, page_size=page)
    return dims, _cache(dims, seqs, width, 5)


def test_token_by_token_is_the_whole_prompt_up_to_growths(gpu_lib):
    dims, cache = _one(width=3, seqs=1)
    _, whole = _one(width=3, seqs=1)
    g = torch.Generator().manual_seed(2)
    v = normal(g, 40, 2, 64) * torch.exp2(torch.randint(-9, 9, (40, 2, 1), generator=g)).bfloat16()
    pos = torch.zeros(40, dtype=torch.int32, device="cuda")
    vd = v.cuda()
    gdn.gdn_kv8_append(dims, None, vd, vd, None, None, None, pos, whole, _ints([0]),
                       cu_seqlens=_ints([0, 40]))
    for t in range(40):
        gdn.gdn_kv8_append(dims, None, vd[t:t + 1], vd[t:t + 1], None, None, None, pos[:1], cache,
                           _ints([t]))
    torch.cuda.synchronize()
    for j in range(2):
        want, once = _kv8.Sequence(64), _kv8.Sequence(64)
        once.append(v[:, j])
        for t in range(40):
            want.append(v[t:t + 1, j])
        assert want.scales == once.scales
        for p in range(40):
            for which in (0, 1):
                assert torch.equal(_row(cache, which, 0, j, p)[0], want.codes[p])
                assert _row(cache, which, 0, j, p)[1] == want.scales[p // 16]
                assert torch.equal(_row(whole, which, 0, j, p)[0], once.codes[p])


def test_a_block_started_anew_and_places_written_again(gpu_lib):
    dims, cache = _one(seqs=1)
    pos = torch.zeros(20, dtype=torch.int32, device="cuda")
    big, small = torch.full((20, 2, 64), 1000.0), torch.full((20, 2, 64), 0.01)
    for x, start, n in ((big, 0, 20), (small, 0, 16)):
        xd = x[:n].bfloat16().cuda()
        gdn.gdn_kv8_append(dims, None, xd, xd, None, None, None, pos[:n], cache, _ints([start]),
                           cu_seqlens=_ints([0, n]))
    # rolled back to 18 tokens, two others there: the scale may only stay or grow
    xd = small[:2].bfloat16().cuda()
    gdn.gdn_kv8_append(dims, None, xd, xd, None, None, None, pos[:2], cache, _ints([18]),
                       cu_seqlens=_ints([0, 2]))
    torch.cuda.synchronize()
    s = float(small.bfloat16()[0, 0, 0])
    assert _row(cache, 0, 0, 0, 3)[1] == 2.0 ** _kv8.exponent(s)
    assert _row(cache, 0, 0, 0, 16)[1] == 2.0 ** _kv8.exponent(1000)
    assert float(_row(cache, 0, 0, 1, 17)[0][0]) == float(_kv8.quantise(
        torch.tensor(1000.0, dtype=torch.float64) / 2.0 ** _kv8.exponent(1000)))
    # 0.01 at a scale of 4 is 1.28 of the smallest steps of 2^-9: one of them
    assert float(_row(cache, 0, 0, 1, 18)[0][0]) == 2.0 ** -9


@pytest.mark.parametrize("x", [0.0, 448.0, 449.0, 448.0 * 2.0 ** 7, 2.0 ** -45, 2.0 ** 90, 1e-38])
def test_borders_of_the_scale(gpu_lib, x):
    dims, cache = _one(seqs=1)
    v = torch.full((1, 2, 64), x).bfloat16()
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv8_append(dims, None, v.cuda(), v.cuda(), None, None, None, pos, cache, _ints([0]))
    torch.cuda.synchronize()
    want = _kv8.Sequence(64)
    want.append(v[0, :1])
    for which in (0, 1):
        codes, scale = _row(cache, which, 0, 0, 0)
        assert scale == want.scales[0] and torch.equal(codes, want.codes[0])


def test_values_that_are_not_finite_stay_in_their_places(gpu_lib):
    dims, cache = _one(seqs=1)
    v = torch.ones(16, 2, 64).bfloat16()
    v[3, 0, 5], v[4, 0, 6], v[5, 1, 7] = math.inf, -math.inf, math.nan
    pos = torch.zeros(16, dtype=torch.int32, device="cuda")
    gdn.gdn_kv8_append(dims, None, v.cuda(), v.cuda(), None, None, None, pos, cache, _ints([0]),
                       cu_seqlens=_ints([0, 16]))
    torch.cuda.synchronize()
    for p in range(16):
        for j in range(2):
            codes, scale = _row(cache, 1, 0, j, p)
            assert scale == 2.0 ** _kv8.exponent(1.0)
            want = v[p, j].double() / scale
            bad = ~torch.isfinite(want)
            assert torch.equal(torch.isnan(codes), bad) and torch.equal(codes[~bad], want[~bad])


def test_padding_and_places_and_pages_that_do_not_exist(gpu_lib):
    dims, cache = _one(seqs=4, width=2, rot=16)
    cache.block_table[3, 0] = 1 << 20
    g = torch.Generator().manual_seed(1)
    x = normal(g, 4, 2, 64).cuda()
    freq = gdn.rope_frequencies(16, 1e4, device="cuda")[0]
    pos = _ints([1, 2, 3, 4])
    before = [t.clone() for t in cache]

    def call(starts, **kw):
        status, k_out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones_like(x)
        q = gdn.gdn_kv8_append(dims, x, x, x, None, None, freq, pos, cache, _ints(starts), k_out=k_out,
                               d_status=status, **kw)
        torch.cuda.synchronize()
        return q, k_out, status.item()
    q, k, status = call([-1, 32, -5, 0])
    assert status == gdn.GDN_DEV_BAD_LENGTH | gdn.GDN_DEV_BAD_PAGE
    for t in (0, 2):
        assert not q[t].any() and not k[t].any()
    plain = gdn.gdn_qk_norm_rope(dims, x, None, None, None, freq, pos)[0]
    assert torch.equal(q[1], plain[1]) and torch.equal(k[3], plain[3])
    for a, b in zip(before, cache):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # ends that are none: nothing is written at all
    for cu in ([0, 3, 2, 4, 4], [1, 2, 3, 4, 4], [0, 1, 2, 3, 5], [0, -1, 2, 3, 4]):
        q = torch.full_like(x, 9)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_kv8_append(dims, x, x, x, None, None, freq, pos, cache, _ints([0, 0, 0, 0]),
                           cu_seqlens=_ints(cu), q_out=q, d_status=status)
        k, v = (torch.full((4, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        gdn.gdn_kv8_gather(dims, cache, _ints(cu), 4, k_out=k, v_out=v, d_status=status)
        torch.cuda.synchronize()
        assert status.item() == gdn.GDN_DEV_BAD_CU_SEQLENS and (q == 9).all() and (k == 9).all()
        for a, b in zip(before, cache):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_gather_of_missing_pages_is_zeros(gpu_lib):
    dims, cache = _one(seqs=2, width=2)
    x = torch.ones(20, 2, 64).bfloat16().cuda()
    pos = torch.zeros(20, dtype=torch.int32, device="cuda")
    gdn.gdn_kv8_append(dims, None, x, x, None, None, None, pos, cache, _ints([0, 0]),
                       cu_seqlens=_ints([0, 20, 20]))
    cache.block_table[0, 1] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = gdn.gdn_kv8_gather(dims, cache, _ints([0, 20, 20]), 20, d_status=status)
    torch.cuda.synchronize()
    assert status.item() == gdn.GDN_DEV_BAD_PAGE
    assert (k[:16] == 1).all() and not k[16:].any() and not v[16:].any()
    status.zero_()
    k, _ = gdn.gdn_kv8_gather(dims, cache, _ints([0, 0, 40]), 40, d_status=status)
    torch.cuda.synchronize()
    assert status.item() & gdn.GDN_DEV_BAD_LENGTH and not k[32:].any()


def test_axes_turn_the_stored_keys(gpu_lib):
    dims, cache = _one(seqs=1, rot=32)
    g = torch.Generator().manual_seed(4)
    x, n = normal(g, 20, 2, 64).cuda(), 20
    freq = gdn.rope_frequencies(32, 1e4, device="cuda")[0]
    pos = torch.randint(0, 900, (3, n), generator=g, dtype=torch.int32).cuda()
    axes = gdn.make_rope_axes(gdn.rope_sections([8, 4, 4], interleaved=True))
    k_out = torch.empty_like(x)
    q = gdn.gdn_kv8_append(dims, x, x, x, None, None, freq, pos, cache, _ints([0]),
                           cu_seqlens=_ints([0, n]), axes=axes, k_out=k_out)
    plain = gdn.gdn_qk_norm_rope_axes(dims, x, None, None, None, freq, pos, axes)[0]
    k, _ = gdn.gdn_kv8_gather(dims, cache, _ints([0, n]), n)
    torch.cuda.synchronize()
    assert torch.equal(q, plain) and torch.equal(k_out, plain)
    err = (k.float() - plain.float()).abs()
    # plain is rounded to bf16, the stored keys from fp32: a half step of each
    assert (err <= (2.0 ** -4 + 2.0 ** -8) * plain.float().abs() + 2.0 ** -10 * 2.0 ** -6).all()
