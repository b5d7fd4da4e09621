"""gdn_kv8_evict: exactly the places that the weights say, ties and NaN among them, at their
new places with their new scales, and nothing else written."""
import math

import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _kv8

pytestmark = pytest.mark.gpu


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _weights(g, kind, n, hkv, cap):
    w = torch.rand(n, hkv, cap, generator=g)
    if kind == "ties":
        return (w * 4).floor() / 4
    if kind == "same":
        return torch.full_like(w, 0.5)
    if kind == "odd":
        w[w < 0.1] = math.nan
        w[(w > 0.1) & (w < 0.2)] = -1.0
        w[(w > 0.2) & (w < 0.25)] = -0.0
        w[(w > 0.25) & (w < 0.27)] = math.inf
        w[(w > 0.27) & (w < 0.3)] = 1e-42
        return w
    return w ** 30 if kind == "small" else w


CASES = [   # lengths, hkv, d, pages from and to (tokens), keep, first, last, weights
    ([1], 1, 64, 16, 1, 0, 0, "any"),
    ([40], 2, 64, 16, 20, 4, 5, "any"),
    ([100, 7, 0, 64, 65], 2, 128, 32, 64, 0, 0, "ties"),
    ([500, 1000], 1, 256, 64, 333, 33, 300, "odd"),       # nothing of the middle
    ([700, 129, 513], 3, 128, 128, 128, 1, 16, "same"),
    ([3000], 4, 256, 64, 1000, 16, 100, "small"),
    ([200] * 60, 2, 64, 16, 199, 0, 1, "odd"),
    ([48, 50], 2, 256, 16, 47, 47, 0, "any"),
    ([9000, 5000], 1, 64, 64, 4096, 0, 0, "ties"),
    ([33_000, 49_153, 8192, 8193], 1, 64, 128, 3000, 7, 200, "odd"),   # more than registers hold
    ([40_000], 1, 64, 128, 1024, 0, 0, "same"),
    ([90], 2, 128, 16, 200, 3, 3, "any"),                 # keeps more than there is
]


@pytest.mark.parametrize("spread", [0.0, 3.0])
@pytest.mark.parametrize("lens,hkv,d,page,keep,first,last,kind", CASES)
def test_evict(gpu_lib, lens, hkv, d, page, keep, first, last, kind, spread):
    g = torch.Generator().manual_seed(sum(lens) + keep)
    n = len(lens)
    cache = _kv8.paged(g, lens, hkv, d, page, spread=spread)
    cap = cache[4].shape[1] * page
    w = _weights(g, kind, n, hkv, cap)
    dims = gdn.make_attn_dims(hkv, hkv, d, page_size=page)
    width = -(-keep // page) + 1
    ids = torch.randperm(n * width + 2, generator=g)[:n * width].to(torch.int32)
    to = gdn.make_kv8_cache(dims, n * width + 2, ids.view(n, width).contiguous().cuda())
    for x in to[:2]:
        x.view(torch.uint8).fill_(0x55)
    for x in to[2:4]:
        x.fill_(-3.0)
    w_out = torch.full((n, hkv, width * page), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    src = gdn.Kv8Cache(*(t.cuda() for t in cache))
    seq_lens, wd = _ints(lens), w.cuda()
    new_lens, kept = gdn.gdn_kv8_evict(dims, src, wd, seq_lens, keep, to, w_out, first=first, last=last,
                                       d_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for t, s in zip(cache, src):   # the source as it was
        assert torch.equal(t.view(torch.uint8), s.cpu().view(torch.uint8))
    assert new_lens.tolist() == [min(v, keep) for v in lens]
    codes = [x.view(torch.uint8).cpu() for x in to[:2]]
    scales = [x.cpu() for x in to[2:4]]
    rows, blocks = torch.zeros(codes[0].shape[:3], dtype=torch.bool), torch.zeros(scales[0].shape, dtype=torch.bool)
    table = to.block_table.cpu()
    for b, length in enumerate(lens):
        for j in range(hkv):
            places = _kv8.evicted(w[b, j], length, keep, first, last)
            m = len(places)
            assert kept[b, j].tolist() == places + [-1] * (keep - m)
            got = w_out[b, j].cpu()
            want = w[b, j, places] if m else w[b, j, :0]
            assert torch.equal(got[:m].view(torch.int32), want.view(torch.int32)) and not got[m:].any()
            if not m:
                continue
            pages = cache[4][b, :-(-length // page)]
            for which in (0, 1):
                c, s = _kv8.of_sequence(cache[which], cache[2 + which], pages, length, j)
                c, s = c[places], s[places]
                for i in range(0, m, 16):
                    top = s[i:i + 16].max()
                    pg, r = int(table[b, i // page]), i % page
                    k = min(16, m - i)
                    rows[pg, j, r:r + k] = True
                    blocks[pg, j, r // 16] = True
                    assert float(scales[which][pg, j, r // 16]) == float(top)
                    want = _kv8.quantise(c[i:i + k] * (s[i:i + k] / top)[:, None])
                    assert torch.equal(codes[which][pg, j, r:r + k].view(_kv8.F8).double(), want)
    for x, s in zip(codes, scales):
        assert (x[~rows] == 0x55).all() and (s[~blocks] == -3.0).all()


def test_pages_that_do_not_exist(gpu_lib):
    g = torch.Generator().manual_seed(1)
    cache = _kv8.paged(g, [64, 64], 1, 64, 16)
    dims = gdn.make_attn_dims(1, 1, 64, page_size=16)
    cache[4][0, 1] = 1 << 29
    src = gdn.Kv8Cache(*(t.cuda() for t in cache))
    w = torch.arange(64.0, device="cuda").expand(2, 1, 64).contiguous()

    def call(lens, bad=False):
        to = gdn.make_kv8_cache(dims, 4, _ints([[0, 1], [2, -1 if bad else 3]]))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        new, kept = gdn.gdn_kv8_evict(dims, src, w, _ints(lens), 32, to, first=20, d_status=status)
        torch.cuda.synchronize()
        return new.tolist(), kept, to, status.item()
    new, kept, to, status = call([64, 64])
    assert status == gdn.GDN_DEV_BAD_PAGE and new == [32, 32]
    assert kept[1, 0].tolist() == [*range(20), *range(52, 64)]
    zero = to.k.view(torch.uint8)[1, 0, :4].any(-1)        # places 16..19 of the missing page
    assert not zero.any() and to.k.view(torch.uint8)[1, 0, 4:].any(-1).all()
    assert call([16, 64], bad=True)[3] == gdn.GDN_DEV_BAD_PAGE
    new, kept, _, status = call([16, 1 << 30])             # longer than the table: cut to it
    assert status == gdn.GDN_DEV_BAD_LENGTH and new == [16, 32]
    assert kept[1, 0].tolist() == [*range(20), *range(52, 64)]


def test_in_a_graph(gpu_lib):
    g = torch.Generator().manual_seed(2)
    lens = [400, 90]
    cache = _kv8.paged(g, lens, 2, 128, 32)
    dims = gdn.make_attn_dims(2, 2, 128, page_size=32)
    src, n = gdn.Kv8Cache(*(t.cuda() for t in cache)), _ints(lens)
    cap = cache[4].shape[1] * 32
    w = torch.rand(2, 2, cap, generator=g).cuda()
    to = gdn.make_kv8_cache(dims, 8, torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4))
    w_out = torch.empty(2, 2, 128, device="cuda")
    new, kept = gdn.gdn_kv8_evict(dims, src, w, n, 100, to, w_out)
    torch.cuda.synchronize()
    want = [x.clone() for x in (new, kept, w_out, to.k.view(torch.uint8), to.v_scale)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_kv8_evict(dims, src, w, n, 100, to, w_out, new_lens=new, kept=kept)
    for x in (new, kept, w_out, to.k.view(torch.uint8), to.v_scale):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (new, kept, w_out, to.k.view(torch.uint8), to.v_scale)):
        assert torch.equal(a, b)
