"""gdn_attn_decode against the 64-bit form (tests/_attn.py has the bound):
lengths of 0 and 1 and around pages, key blocks and the runs that CTAs share,
every head dim, 16-bit type, page size and group size (above 16 too), shared
prefixes with rows shorter than the prefix, whatever the cache holds beyond a
sequence, bad pages and lengths, strided views, other streams, graphs, and the
whole layer step by step against the prefill."""
import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _attn
from tests._attn import IO, normal

pytestmark = pytest.mark.gpu


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _workspace(dims, n, shared):
    # whatever an earlier call left there must not matter: NaN bytes
    size = gdn.gdn_attn_decode_workspace_size(dims, n, shared)
    return torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")


CASES = [   # lengths, hq, hkv, d, page, io, gate, shared
    ([1], 2, 1, 64, 16, "bf16", False, 0),
    ([1], 16, 4, 256, 64, "bf16", True, 0),
    ([700], 16, 4, 256, 64, "bf16", True, 0),
    ([5000], 4, 2, 128, 128, "fp16", False, 0),
    ([0, 1, 0, 63, 64, 65, 0], 4, 2, 256, 64, "bf16", True, 0),
    ([15, 16, 17, 33, 300], 4, 1, 128, 16, "bf16", False, 0),
    ([127, 128, 129, 1000, 2], 6, 2, 64, 128, "fp16", True, 0),
    ([31, 32, 500], 3, 3, 256, 32, "fp16", False, 0),
    ([100, 7], 40, 2, 128, 64, "bf16", True, 0),          # groups of twenty: two items
    ([200, 90], 16, 1, 256, 16, "bf16", False, 0),
    (list(range(1, 400, 9)), 4, 2, 64, 32, "bf16", False, 0),
    ([0, 0, 0], 4, 2, 128, 32, "bf16", True, 0),
    ([320, 257, 300], 4, 2, 256, 64, "bf16", True, 256),
    ([16, 16], 2, 1, 128, 16, "bf16", False, 16),         # nothing beyond the prefix
    ([145, 200, 144], 6, 2, 128, 16, "fp16", True, 144),  # a prefix that ends inside a block
    ([1000, 640, 3, 0, 641], 4, 2, 256, 128, "bf16", False, 640),   # rows inside the prefix
    ([2100, 2050], 16, 1, 64, 32, "bf16", True, 2048),
    ([400] * 70, 4, 2, 64, 64, "fp16", False, 320),       # more than one row block of the prefix
    ([300, 310], 40, 2, 256, 32, "bf16", False, 288),
    ([90], 4, 1, 128, 16, "bf16", True, 64),              # one row: no prefix pass
]


@pytest.mark.parametrize("lens,hq,hkv,d,page,io,gate,shared", CASES)
def test_decode(gpu_lib, lens, hq, hkv, d, page, io, gate, shared):
    g = torch.Generator().manual_seed(sum(lens) + d)
    dt, n = IO[io], len(lens)
    kc, vc, table = _attn.paged(g, lens, hkv, d, page, dt, shared=shared)
    qg = normal(g, n, hq, 2 * d, dtype=dt)
    dims = gdn.make_attn_dims(hq, hkv, d, io=io, page_size=page)
    qgd, status = qg.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    # rows that end inside the prefix see its first tokens
    ref, slack = _attn.decode(qg[..., :d], kc, vc, table, lens, qg[..., d:] if gate else None,
                              _attn.scale_of(d), dt)
    # a block table that could hold long sequences, its other entries no pages at all:
    # the form for few keys does not apply
    wide = torch.full((n, max(table.shape[1], 16384 // page)), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    for what, tb in (("o", table), ("o (wide table)", wide)):
        o = gdn.gdn_attn_decode(dims, qgd[..., :d], kc.cuda(), vc.cuda(), tb.cuda(), _ints(lens),
                                _workspace(dims, n, shared), shared_len=shared,
                                gate=qgd[..., d:] if gate else None, d_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        _attn.check(o, ref, slack, dt, what)


def test_growing_scores_and_scale(gpu_lib):
    g = torch.Generator().manual_seed(12)
    lens, d, page = [900, 130], 128, 64
    kc, vc, table = _attn.paged(g, lens, 1, d, page, torch.bfloat16)
    for b, length in enumerate(lens):
        for t in range(length):
            kc[table[b, t // page].long(), :, t % page] *= 8.0 * t / length
    q = normal(g, 2, 2, d)
    dims = gdn.make_attn_dims(2, 1, d, page_size=page, scale=0.5)
    o = gdn.gdn_attn_decode(dims, q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), _ints(lens),
                            _workspace(dims, 2, 0))
    ref, slack = _attn.decode(q, kc, vc, table, lens, None, 0.5, torch.bfloat16)
    _attn.check(o, ref, slack, torch.bfloat16, "o")


def test_bad_pages_and_lengths_are_reported(gpu_lib):
    g = torch.Generator().manual_seed(1)
    d, page, lens = 128, 16, [40, 33, 20]
    kc, vc, table = _attn.paged(g, lens, 1, d, page, torch.bfloat16)
    q = normal(g, 3, 2, d)
    dims = gdn.make_attn_dims(2, 1, d, page_size=page)

    def call(tb, ln, shared=0):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = gdn.gdn_attn_decode(dims, q.cuda(), kc.cuda(), vc.cuda(), tb.cuda(), _ints(ln),
                                _workspace(dims, 3, shared), shared_len=shared, d_status=status)
        torch.cuda.synchronize()
        return o, status.item()
    good, status = call(table, lens)
    assert status == 0
    for bad in (kc.shape[0], -1, 2 ** 31 - 1):
        t2 = table.clone()
        t2[1, 2] = bad
        o, status = call(t2, lens)
        assert status == gdn.GDN_DEV_BAD_PAGE
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])   # the other rows stand
        t2 = table.clone()
        t2[0, 0] = bad
        assert call(t2, lens, shared=16)[1] == gdn.GDN_DEV_BAD_PAGE
    # entries past a row's length are not looked at
    t2 = table.clone()
    t2[2, 2] = 2 ** 31 - 1
    o, status = call(t2, lens)
    assert status == 0 and torch.equal(o, good)
    # a length that the block table cannot hold is cut to what it holds
    _, status = call(table, [40, 33, 49])
    assert status == gdn.GDN_DEV_BAD_LENGTH
    o, status = call(table, [40, 33, -7])
    assert status == 0 and (o[2] == 0).all() and torch.equal(o[:2], good[:2])


@pytest.mark.parametrize("shared", [0, 1024])
def test_long_ragged_batch_matches_a_float32_form_and_repeats(gpu_lib, shared):
    g = torch.Generator(device="cuda").manual_seed(7)
    n, hq, hkv, d, page = 23, 16, 4, 256, 64
    lens = [shared + 1 + (i * 977) % 3000 for i in range(n)]
    width = max(lens) // page + 1
    pool = n * width
    table = torch.randperm(pool, generator=g, device="cuda").to(torch.int32).view(n, width)
    table[:, :shared // page] = table[0, :shared // page].clone()
    kc, vc = (torch.randn(pool, hkv, page, d, generator=g, device="cuda").to(torch.bfloat16)
              for _ in range(2))
    q = torch.randn(n, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    dims = gdn.make_attn_dims(hq, hkv, d, page_size=page)
    ws = _workspace(dims, n, shared)
    o = gdn.gdn_attn_decode(dims, q, kc, vc, table, _ints(lens), ws, shared_len=shared)
    again = gdn.gdn_attn_decode(dims, q, kc, vc, table, _ints(lens), ws, shared_len=shared)
    assert torch.equal(o, again)
    ref = torch.empty(n, hq, d, device="cuda")
    for b, length in enumerate(lens):
        k, v = (c[table[b].long()].transpose(0, 1).reshape(hkv, -1, d)[:, :length].float()
                for c in (kc, vc))
        s = q[b].float().view(hkv, -1, d) @ k.transpose(1, 2) / 16
        ref[b] = (torch.softmax(s, -1) @ v).reshape(hq, d)
    assert float((o.float() - ref).norm() / ref.norm()) < 2 * 2.0 ** -8


def test_on_another_stream_and_from_a_graph(gpu_lib):
    g = torch.Generator().manual_seed(15)
    lens, hq, hkv, d, page, shared = [300, 150, 129], 4, 2, 256, 64, 128
    kc, vc, table = _attn.paged(g, lens, hkv, d, page, torch.bfloat16, shared=shared)
    kc, vc, table, ln = kc.cuda(), vc.cuda(), table.cuda(), _ints(lens)
    q = normal(g, 3, hq, d).cuda()
    dims = gdn.make_attn_dims(hq, hkv, d, page_size=page)
    ws = _workspace(dims, 3, shared)

    def call(o=None):
        return gdn.gdn_attn_decode(dims, q, kc, vc, table, ln, ws, shared_len=shared, o=o)
    plain = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o = call()
    side.synchronize()
    assert torch.equal(o, plain)
    o = torch.zeros_like(plain)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        call(o)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, plain)
    # a replay follows the lengths that are in the buffer by then
    ln.copy_(_ints([200, 150, 1]))
    graph.replay()
    torch.cuda.synchronize()
    ref, slack = _attn.decode(q.cpu(), kc.cpu(), vc.cpu(), table.cpu(), [200, 150, 1], None,
                              _attn.scale_of(d), torch.bfloat16)
    _attn.check(o, ref, slack, torch.bfloat16, "o")


def test_appending_and_decoding_token_by_token_equals_the_prefill(gpu_lib):
    """A prompt through gdn_qk_norm_rope and gdn_attn_prefill, and the same
    tokens one by one through gdn_kv_append and gdn_attn_decode: equal up to
    the rounding of weights and outputs of either."""
    g = torch.Generator().manual_seed(33)
    n, hq, hkv, d, page = 70, 8, 2, 256, 16
    qg, kv = normal(g, n, hq, 2 * d).cuda(), normal(g, n, 2 * hkv, d).cuda()
    q, gate, k, v = qg[..., :d], qg[..., d:], kv[:, :hkv], kv[:, hkv:]
    w = 1 + 0.1 * torch.randn(d, generator=g).cuda()
    freq = gdn.rope_frequencies(64, 1e6, device="cuda")[0]
    dims = gdn.make_attn_dims(hq, hkv, d, rot_dim=64, page_size=page)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    qn, kn = gdn.gdn_qk_norm_rope(dims, q, k, w, w, freq, pos)
    full = gdn.gdn_attn_prefill(dims, qn, kn, v, _ints([0, n]), gate=gate)
    kc = torch.full((6, hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc, table = kc.clone(), _ints([[4, 0, 5, 1, 3]])
    ws = _workspace(dims, 1, 0)
    for t in range(n):
        one = slice(t, t + 1)
        qt = gdn.gdn_kv_append(dims, q[one], k[one], v[one], w, w, freq, pos[one], kc, vc, table)
        assert torch.equal(qt, qn[one])
        o = gdn.gdn_attn_decode(dims, qt, kc, vc, table, _ints([t + 1]), ws, gate=gate[one])
        err = (o.float() - full[one].float()).abs().max()
        assert float(err) <= 4 * 2.0 ** -8 * float(v.float().abs().max()), t


def test_a_cache_past_32_bit_offsets(gpu_lib):
    """Rows beyond 2^31 elements of the pool: appended, then read back by decode,
    alone (few keys) and behind a shared prefix."""
    g = torch.Generator().manual_seed(44)
    hq, hkv, d, page = 2, 1, 256, 128
    pool = 2 ** 31 // (hkv * page * d) + 40
    kc = torch.empty(pool, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    lens = [300, 290]
    rows = sum(lens)
    assert (pool - 8) * hkv * page * d > 2 ** 31
    table = torch.tensor([[pool - 1, pool - 5, pool - 2], [pool - 1, pool - 3, pool - 4]],
                         dtype=torch.int32)
    k, v = normal(g, rows, hkv, d), normal(g, rows, hkv, d)
    k[300:428], v[300:428] = k[:128], v[:128]           # the first page is common
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    seq = torch.tensor([0] * 300 + [1] * 290, dtype=torch.int32)
    pos[300:428] = -1                                    # and written once
    dims = gdn.make_attn_dims(hq, hkv, d, page_size=page)
    gdn.gdn_kv_append(dims, None, k.cuda(), v.cuda(), None, None, None, pos.cuda(), kc, vc,
                      table.cuda(), row_seq=seq.cuda())
    q = normal(g, 2, hq, d)
    last = kc[pool - 8:].cpu(), vc[pool - 8:].cpu()
    ref, slack = _attn.decode(q, *last, table - (pool - 8), lens, None, _attn.scale_of(d),
                              torch.bfloat16)
    for shared in (0, 128):
        o = gdn.gdn_attn_decode(dims, q.cuda(), kc, vc, table.cuda(), _ints(lens),
                                _workspace(dims, 2, shared), shared_len=shared)
        _attn.check(o, ref, slack, torch.bfloat16, f"shared {shared}")


@pytest.mark.parametrize("lens,hq,hkv,d,page,gate,shared", [
    ([9000], 24, 2, 256, 64, True, 0),            # twelve rows an item
    ([5000, 1], 10, 2, 64, 64, False, 0),         # five
    ([4100, 0, 4097], 20, 1, 128, 32, True, 0),   # sixteen and four
    ([6000, 3000], 7, 7, 64, 128, True, 0),       # one
    ([3000, 2200, 2048], 36, 2, 128, 16, True, 2048),
])
def test_few_long_sequences(gpu_lib, lens, hq, hkv, d, page, gate, shared):
    """Items cut into many runs, their rows and partials joined by many CTAs."""
    g = torch.Generator().manual_seed(sum(lens) + hq)
    dt, n = torch.bfloat16, len(lens)
    kc, vc, table = _attn.paged(g, lens, hkv, d, page, dt, shared=shared)
    qg = normal(g, n, hq, 2 * d, dtype=dt).cuda()
    dims = gdn.make_attn_dims(hq, hkv, d, page_size=page)
    o = gdn.gdn_attn_decode(dims, qg[..., :d], kc.cuda(), vc.cuda(), table.cuda(), _ints(lens),
                            _workspace(dims, n, shared), shared_len=shared,
                            gate=qg[..., d:] if gate else None)
    qc = qg.cpu()
    ref, slack = _attn.decode(qc[..., :d], kc, vc, table, lens, qc[..., d:] if gate else None,
                              _attn.scale_of(d), dt)
    _attn.check(o, ref, slack, dt, "o")
