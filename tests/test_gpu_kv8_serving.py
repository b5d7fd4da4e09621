"""The 8-bit cache's calls together, as a server makes them: prompts with positions of
several axes go in, their second chunk attends to what the cache gives back, tokens are
decoded while their attention is counted, the sequences are cut down by it and go
on in other pages.  Every step is checked in 64 bits against what the one before it
left on the device.  And what the calls allow besides: other streams, outputs in
place, graphs, pools past 32 bits, waits that run out."""
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


def _host(cache):
    return tuple(x.cpu() for x in cache)


def _spread(n, width, pool, seed):
    ids = torch.randperm(pool, generator=torch.Generator().manual_seed(seed))[:n * width]
    return ids.to(torch.int32).view(n, width).contiguous().cuda()


@pytest.mark.parametrize("prompts,hq,hkv,d,rot,page,io,inter", [
    ([[70, 5, 1], [30, 90, 17]], 8, 2, 128, 128, 16, "bf16", True),
    ([[129, 40], [1, 64]], 16, 1, 256, 64, 64, "bf16", False),
    ([[33, 0, 200, 8], [20, 12, 1, 150]], 6, 3, 64, 32, 32, "fp16", True),
])
def test_prompts_to_decoding_to_eviction_and_on(gpu_lib, prompts, hq, hkv, d, rot, page, io, inter):
    g = torch.Generator().manual_seed(d + sum(prompts[0]))
    dt, n = IO[io], len(prompts[0])
    dims = gdn.make_attn_dims(hq, hkv, d, io=io, rot_dim=rot, page_size=page)
    scale, steps, keep = _attn.scale_of(d), 3, 40
    longest = max(sum(p) for p in zip(*prompts)) + steps
    width = -(-longest // page)
    cache = gdn.make_kv8_cache(dims, n * width + 3, _spread(n, width, n * width + 3, d))
    sections = [rot // 2 - 2 * (rot // 8), rot // 8, rot // 8]
    axes = gdn.make_rope_axes(gdn.rope_sections(sections, interleaved=inter))
    freq, factor = gdn.rope_frequencies(rot, 1e6, device="cuda")
    norms = [(1 + 0.1 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    held = [0] * n

    def append(c, rows, starts, cu):
        qg, kv = normal(g, rows, hq, 2 * d, dtype=dt), normal(g, rows, 2 * hkv, d, dtype=dt)
        pos = torch.randint(0, 5000, (3, rows), generator=g, dtype=torch.int32)
        qd, kvd = qg.cuda(), kv.cuda()
        q = gdn.gdn_kv8_append(dims, qd[..., :d], kvd[:, :hkv], kvd[:, hkv:], *norms, freq, pos.cuda(), c,
                               _ints(starts), cu_seqlens=cu, axes=axes, rope_scale=factor,
                               d_status=status)
        plain, _ = gdn.gdn_qk_norm_rope_axes(dims, qd[..., :d].contiguous(), kvd[:, :hkv].contiguous(),
                                             *norms, freq, pos.cuda(), axes, rope_scale=factor)
        assert torch.equal(q, plain)
        return q, qd[..., d:], qg[..., d:]

    for rows in prompts:
        cu = _ends(rows)
        q, gate, gate_h = append(cache, cu[-1], held, _ints(cu))
        held = [a + b for a, b in zip(held, rows)]
        cu_kv = _ends(held)
        k, v = gdn.gdn_kv8_gather(dims, cache, _ints(cu_kv), cu_kv[-1], d_status=status)
        host = _host(cache)
        for b in range(n):
            for j in range(hkv):
                pages = host[4][b, :-(-held[b] // page)]
                for got, which in ((k, 0), (v, 1)):
                    codes, scales = _kv8.of_sequence(host[which], host[2 + which], pages, held[b], j)
                    assert torch.equal(got[cu_kv[b]:cu_kv[b + 1], j].cpu(), (codes * scales[:, None]).to(dt))
        o = gdn.gdn_attn_prefill(dims, q, k, v, _ints(cu), _ints(cu_kv), gate=gate, d_status=status)
        ref, slack = _attn.prefill(q.cpu(), k.cpu(), v.cpu(), cu, cu_kv, gate_h, scale, dt)
        _attn.check(o, ref, slack, dt, f"prompt {rows}")

    weights = torch.zeros(n, hkv, width * page, device="cuda")

    def decode(c, lens, w):
        q, gate, gate_h = append(c, n, lens, None)
        lens = [x + 1 for x in lens]
        ws = torch.empty(gdn.gdn_attn_decode_kv8_workspace_size(dims, n, w.shape[2]), dtype=torch.uint8,
                         device="cuda")
        old = w.clone()
        o = gdn.gdn_attn_decode_kv8(dims, q, c, _ints(lens), ws, gate=gate, weights=w, d_status=status)
        ref, slack, dw, dws = _kv8.decode(q.cpu(), _host(c), lens, gate_h, scale, dt)
        _attn.check(o, ref, slack, dt, f"decode at {lens}")
        _kv8.check_weights(w, old, dw, dws, f"weights at {lens}")
        return lens

    for _ in range(steps):
        held = decode(cache, held, weights)

    small = -(-(keep + steps) // page)
    to = gdn.make_kv8_cache(dims, n * small + 1, _spread(n, small, n * small + 1, 7))
    out = torch.full((n, hkv, small * page), 9.0, device="cuda")
    lens, kept = gdn.gdn_kv8_evict(dims, cache, weights, _ints(held), keep, to, weights_out=out, first=4,
                                   last=8, d_status=status)
    assert lens.tolist() == [min(x, keep) for x in held]
    a, b = _host(cache), _host(to)
    for s in range(n):
        for j in range(hkv):
            want = _kv8.evicted(weights[s, j], held[s], keep, 4, 8)
            assert kept[s, j].tolist() == want + [-1] * (keep - len(want))
            assert torch.equal(out[s, j, :len(want)].cpu(), weights[s, j].cpu()[want])
            assert not out[s, j, len(want):].any()
            for which in range(2):
                c, sc = _kv8.of_sequence(a[which], a[2 + which], a[4][s], held[s], j)
                c2, s2 = _kv8.of_sequence(b[which], b[2 + which], b[4][s], len(want), j)
                pad = -len(want) % 16
                top = torch.cat([sc[want], torch.zeros(pad, dtype=torch.float64)]).view(-1, 16).amax(1)
                top = top.repeat_interleave(16)[:len(want)]
                assert torch.equal(s2, top)
                assert torch.equal(c2, _kv8.quantise(c[want] * (sc[want] / top)[:, None]))
    held = lens.tolist()
    for _ in range(steps):
        held = decode(to, held, out)
    assert status.item() == 0


def _calls():
    """Each call with its outputs left to it, as a function of the stream."""
    g = torch.Generator().manual_seed(3)
    n, hq, hkv, d, page = 640, 4, 2, 128, 64
    dims = gdn.make_attn_dims(hq, hkv, d, rot_dim=64, page_size=page)
    q, k, v = (normal(g, n, h, d).cuda() for h in (hq, hkv, hkv))
    w, freq = torch.ones(d, device="cuda"), gdn.rope_frequencies(64, 1e6, device="cuda")[0]
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    table = torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1)
    zeros = torch.zeros(n, dtype=torch.int32, device="cuda")
    full = torch.full((n,), page, dtype=torch.int32, device="cuda")
    cache, other, to = (gdn.make_kv8_cache(dims, n, table) for _ in range(3))
    cu = page * torch.arange(n + 1, dtype=torch.int32, device="cuda")
    rows = [normal(g, n * page, h, d).cuda() for h in (hkv, hkv)]
    gdn.gdn_kv8_append(dims, None, *rows, None, None, freq, cu[:1].expand(n * page).contiguous(), cache,
                       zeros, cu_seqlens=cu)
    ws = torch.empty(gdn.gdn_attn_decode_kv8_workspace_size(dims, n), dtype=torch.uint8, device="cuda")
    weights = torch.rand(n, hkv, page, generator=g).cuda()
    axes, pos3 = gdn.make_rope_axes(gdn.rope_sections([16, 8, 8])), pos.expand(3, n).contiguous()
    return {"axes": lambda **s: gdn.gdn_qk_norm_rope_axes(dims, q, k, w, w, freq, pos3, axes, **s)[0],
            "append": lambda **s: gdn.gdn_kv8_append(dims, q, k, v, w, w, freq, pos, other, zeros, **s),
            "gather": lambda **s: gdn.gdn_kv8_gather(dims, cache, cu, n * page, **s)[1],
            "decode": lambda **s: gdn.gdn_attn_decode_kv8(dims, q, cache, full, ws, **s),
            "evict": lambda **s: gdn.gdn_kv8_evict(dims, cache, weights, full, 48, to, **s)[1]}


@pytest.mark.parametrize("name", ["axes", "append", "gather", "decode", "evict"])
def test_work_that_the_current_stream_still_has_to_do_stays_out(gpu_lib, name):
    call = _calls()[name]
    plain = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    was = torch.empty_like(plain)     # freed with a write to it still to come
    torch.cuda._sleep(100_000_000)
    was.fill_(7)
    del was
    o = call(stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(o, plain)
    spans = [(s["address"], s["address"] + s["total_size"], s["stream"])
             for s in torch.cuda.memory_snapshot()]
    assert [s for a, b, s in spans if a <= o.data_ptr() < b] == [side.cuda_stream]


@pytest.mark.parametrize("name", ["axes", "append", "gather", "decode", "evict"])
def test_captured_and_replayed(gpu_lib, name):
    call = _calls()[name]
    plain = call().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = call()
    for _ in range(3):
        o.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, plain)


# few rows, and whole blocks enough for the ring of tiles
@pytest.mark.parametrize("lens", [[3, 40], [2600, 1, 30]])
@pytest.mark.parametrize("d", [64, 256])
def test_append_in_place(gpu_lib, lens, d):
    g = torch.Generator().manual_seed(sum(lens))
    n, hq, hkv, page = sum(lens), 4, 2, 32
    dims = gdn.make_attn_dims(hq, hkv, d, rot_dim=64, page_size=page)
    q, k, v = (normal(g, n, h, d).cuda() for h in (hq, hkv, hkv))
    w, freq = torch.ones(d, device="cuda"), gdn.rope_frequencies(64, 1e6, device="cuda")[0]
    width = -(-max(lens) // page) + 1
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    runs = []
    for place in (False, True):
        cache = gdn.make_kv8_cache(dims, len(lens) * width, _spread(len(lens), width, len(lens) * width, 1))
        a, b = q.clone(), k.clone()
        k_out = b if place else torch.empty_like(k)
        o = gdn.gdn_kv8_append(dims, a, b, v, w, w, freq, pos, cache, _ints([0] * len(lens)),
                               cu_seqlens=_ints(_ends(lens)), q_out=a if place else None, k_out=k_out)
        runs.append([o, k_out, *[x.view(torch.uint8) for x in cache[:2]], *cache[2:]])
    assert runs[1][0].data_ptr() != runs[0][0].data_ptr()
    for x, y in zip(*runs):
        assert torch.equal(x, y)


def test_a_pool_past_32_bits(gpu_lib):
    """The same sequences in the first and in the last pages of a pool of 5 GB each of k and v."""
    g = torch.Generator().manual_seed(8)
    hq, hkv, d, page, pool, lens = 16, 8, 256, 128, 20000, [700, 40, 3]
    dims = gdn.make_attn_dims(hq, hkv, d, rot_dim=64, page_size=page)
    n, width, rows = len(lens), 6, sum(lens)
    first = torch.arange(n * width, dtype=torch.int32, device="cuda").view(n, width)
    cache = gdn.make_kv8_cache(dims, pool, first)
    freq = gdn.rope_frequencies(64, 1e6, device="cuda")[0]
    q, k, v = (normal(g, rows, h, d).cuda() for h in (hq, hkv, hkv))
    pos, cu, ln = torch.arange(rows, dtype=torch.int32, device="cuda"), _ints(_ends(lens)), _ints(lens)
    ws = torch.empty(gdn.gdn_attn_decode_kv8_workspace_size(dims, n, width * page), dtype=torch.uint8,
                     device="cuda")
    results = []
    for at in (0, pool - 4 * n * width):
        c = cache._replace(block_table=first + at)
        to = cache._replace(block_table=first + at + 2 * n * width)
        gdn.gdn_kv8_append(dims, q, k, v, None, None, freq, pos, c, _ints([0] * n), cu_seqlens=cu)
        w = torch.zeros(n, hkv, width * page, device="cuda")
        o = gdn.gdn_attn_decode_kv8(dims, q[:n], c, ln, ws, weights=w)
        new, kept = gdn.gdn_kv8_evict(dims, c, w, ln, 100, to)
        cu2 = torch.cat([_ints([0]), new.cumsum(0, dtype=torch.int32)])
        o2 = gdn.gdn_attn_decode_kv8(dims, q[:n], to, new, ws)
        results.append([o, w, new, kept, o2, *gdn.gdn_kv8_gather(dims, c, cu, rows),
                        *gdn.gdn_kv8_gather(dims, to, cu2, int(cu2[-1]))])
    for x, y in zip(*results):
        assert torch.equal(x, y)
    assert results[0][5].any()


@pytest.mark.parametrize("lens,hq,hkv,d", [([2600], 4, 2, 256), ([1500, 1300], 12, 3, 64),
                                           ([2500], 24, 1, 128)])
def test_an_append_whose_wait_runs_out(gpu_lib, lens, hq, hkv, d):
    g = torch.Generator().manual_seed(d)
    rows, n, page = sum(lens), len(lens), 64
    width = -(-max(lens) // page)
    table = torch.arange(n * width, dtype=torch.int32, device="cuda").view(n, width)
    q, k, v = (normal(g, rows, h, d).cuda() for h in (hq, hkv, hkv))
    freq = gdn.rope_frequencies(64, 1e6, device="cuda")[0]
    pos, cu = torch.arange(rows, dtype=torch.int32, device="cuda"), _ints(_ends(lens))

    def call(flags):
        dims = gdn.make_attn_dims(hq, hkv, d, rot_dim=64, page_size=page, flags=flags)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        cache = gdn.make_kv8_cache(dims, n * width, table)
        o = gdn.gdn_kv8_append(dims, q, k, v, None, None, freq, pos, cache, _ints([0] * n), cu_seqlens=cu,
                               q_out=torch.full_like(q, 7.0), d_status=status)
        torch.cuda.synchronize()
        return o, cache, status.item()
    o, cache, status = call(0)
    assert status == 0
    o2, cache2, status = call(gdn.GDN_TEST_WAIT_TIMEOUT)
    assert status == gdn.GDN_DEV_WAIT_TIMEOUT
    assert (o2[:16, 0] == 7).all()
    assert torch.equal(o2[16:], o[16:])       # rows of the other blocks
    for x, y in zip(cache[:2], cache2[:2]):
        assert torch.equal(x.view(torch.uint8)[0, :, 16:], y.view(torch.uint8)[0, :, 16:])
        assert torch.equal(x.view(torch.uint8)[1:], y.view(torch.uint8)[1:])
    o, _, status = call(0)
    assert status == 0 and not (o[:16] == 7).all()


def test_two_streams_at_once(gpu_lib):
    """Steps of two batches on two streams, each with its workspace, many times."""
    g = torch.Generator().manual_seed(5)
    sets = []
    for hq, hkv, d, lens in ((16, 4, 256, [900, 2000, 30, 1]), (8, 8, 64, [3000] * 20)):
        dims = gdn.make_attn_dims(hq, hkv, d, page_size=64)
        k8, v8, ks, vs, table = _kv8.paged(g, lens, hkv, d, 64)
        cache = gdn.Kv8Cache(*[x.cuda() for x in (k8, v8, ks, vs, table)])
        cap = table.shape[1] * 64
        ws = torch.empty(gdn.gdn_attn_decode_kv8_workspace_size(dims, len(lens), cap), dtype=torch.uint8,
                         device="cuda")
        q, w = normal(g, len(lens), hq, d).cuda(), torch.zeros(len(lens), hkv, cap, device="cuda")
        o = gdn.gdn_attn_decode_kv8(dims, q, cache, _ints(lens), ws, weights=w)
        sets.append((dims, q, cache, _ints(lens), ws, w, o, w.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, (dims, q, cache, lens, ws, w, _, _, s) in enumerate(sets):
            with torch.cuda.stream(s):
                w.zero_()
                outs[i].append((gdn.gdn_attn_decode_kv8(dims, q, cache, lens, ws, weights=w), w.clone()))
    torch.cuda.synchronize()
    for i, s in enumerate(sets):
        for o, w in outs[i]:
            assert torch.equal(o, s[6]) and torch.equal(w, s[7])
