"""gdn_attn_prefill against the 64-bit form (tests/_attn.py has the bound):
sequences of 0 and 1 tokens to several row and key blocks and the sizes around
a block, every head dim, 16-bit type and group size, more and fewer keys than
queries (rows that see nothing), strided views, gates, what lies in other
sequences, large scores, refused cu_seqlens, other streams, graphs."""
import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _attn
from tests._attn import IO, normal

pytestmark = pytest.mark.gpu


def _cu(lens):
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    return cu


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _run(dims, q, k, v, cu_q, cu_kv=None, gate=None, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = gdn.gdn_attn_prefill(dims, q, k, v, _ints(cu_q), None if cu_kv is None else _ints(cu_kv),
                             gate=gate, d_status=status, **kw)
    torch.cuda.synchronize()
    assert status.item() == 0
    return o


CASES = [   # queries, keys (None: the same), hq, hkv, d, io, gate
    ([1], None, 2, 1, 64, "bf16", False),
    ([1], None, 4, 2, 128, "bf16", True),
    ([1], None, 4, 1, 256, "fp16", False),
    ([5], None, 4, 1, 256, "bf16", True),
    ([63, 1, 64, 65], None, 4, 2, 128, "fp16", True),
    ([127, 128, 129], None, 2, 2, 64, "bf16", False),
    ([255, 257], None, 1, 1, 256, "bf16", False),
    ([0, 300, 0, 0, 41, 0], None, 4, 2, 256, "bf16", True),
    ([130, 7], None, 6, 2, 128, "bf16", True),        # groups of three
    ([90], None, 12, 1, 64, "fp16", False),           # groups of twelve: three of four
    ([40, 33], None, 16, 1, 128, "bf16", False),      # sixteen heads to a block
    ([33], None, 128, 1, 64, "bf16", False),          # a whole block of heads
    ([700], None, 2, 1, 128, "bf16", False),
    ([520], None, 2, 1, 256, "fp16", True),
    ([600], None, 1, 1, 64, "bf16", False),
    ([3, 17, 1], [200, 17, 129], 4, 2, 256, "bf16", False),   # more keys than queries
    ([1, 1], [384, 1000], 2, 1, 128, "fp16", False),
    ([20, 140, 3], [5, 130, 0], 4, 2, 128, "bf16", True),     # first rows see nothing
    ([150, 2], [0, 0], 2, 2, 256, "bf16", False),             # no key at all
    ([130], [131], 2, 1, 64, "fp16", False),
]


@pytest.mark.parametrize("lens_q,lens_kv,hq,hkv,d,io,gate", CASES)
def test_prefill(gpu_lib, lens_q, lens_kv, hq, hkv, d, io, gate):
    g = torch.Generator().manual_seed(sum(lens_q) + 7 * d)
    dt = IO[io]
    cu_q = _cu(lens_q)
    cu_kv = cu_q if lens_kv is None else _cu(lens_kv)
    # q beside its gate, k beside v, as a projection leaves them
    qg, kv = normal(g, cu_q[-1], hq, 2 * d, dtype=dt), normal(g, cu_kv[-1], 2 * hkv, d, dtype=dt)
    q, gt, k, v = qg[..., :d], qg[..., d:] if gate else None, kv[:, :hkv], kv[:, hkv:]
    dims = gdn.make_attn_dims(hq, hkv, d, io=io)
    qgd, kvd = qg.cuda(), kv.cuda()
    o = _run(dims, qgd[..., :d], kvd[:, :hkv], kvd[:, hkv:], cu_q,
             None if lens_kv is None else cu_kv, qgd[..., d:] if gate else None)
    ref, slack = _attn.prefill(q, k, v, cu_q, cu_kv, gt, _attn.scale_of(d), dt)
    _attn.check(o, ref, slack, dt, "o")


def test_scale_and_large_scores(gpu_lib):
    """Scores of several hundred: the running maximum rises block after block
    (later keys are larger), so the accumulated output is rescaled."""
    g = torch.Generator().manual_seed(8)
    n, hq, hkv, d = 650, 2, 1, 128
    q, v = normal(g, n, hq, d), normal(g, n, hkv, d)
    k = (normal(g, n, hkv, d).float() * torch.linspace(0.05, 6, n)[:, None, None]).to(torch.bfloat16)
    dims = gdn.make_attn_dims(hq, hkv, d, scale=0.7)
    o = _run(dims, q.cuda(), k.cuda(), v.cuda(), [0, n])
    scale = float(torch.tensor(0.7, dtype=torch.float32))
    ref, slack = _attn.prefill(q, k, v, [0, n], [0, n], None, scale, torch.bfloat16)
    _attn.check(o, ref, slack, torch.bfloat16, "o")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_other_sequences_never_reach_a_sequence(gpu_lib, d, bad):
    g = torch.Generator().manual_seed(4)
    lens = [70, 150, 60, 129]
    cu, hq, hkv = _cu(lens), 2, 1
    q, k, v = (normal(g, cu[-1], h, d) for h in (hq, hkv, hkv))
    for t in (q, k, v):
        t[cu[0]:cu[1]] = bad
        t[cu[2]:cu[3]] = bad
    dims = gdn.make_attn_dims(hq, hkv, d)
    o = _run(dims, q.cuda(), k.cuda(), v.cuda(), cu).cpu()
    for b in (1, 3):
        rows = slice(cu[b], cu[b + 1])
        ref, slack = _attn.prefill(q[rows], k[rows], v[rows], [0, lens[b]], [0, lens[b]], None,
                                   _attn.scale_of(d), torch.bfloat16)
        _attn.check(o[rows], ref, slack, torch.bfloat16, f"sequence {b}")


def test_nan_keys_reach_the_rows_that_see_them_only(gpu_lib):
    g = torch.Generator().manual_seed(14)
    n, d = 300, 128
    q, k, v = (normal(g, n, 1, d) for _ in range(3))
    k[200] = float("nan")
    o = _run(gdn.make_attn_dims(1, 1, d), q.cuda(), k.cuda(), v.cuda(), [0, n]).cpu()
    assert torch.isnan(o[200:]).all() and torch.isfinite(o[:200]).all()
    ref, slack = _attn.prefill(q[:200], k[:200], v[:200], [0, 200], [0, 200], None,
                               _attn.scale_of(d), torch.bfloat16)
    _attn.check(o[:200], ref, slack, torch.bfloat16, "rows before it")


def test_bad_cu_seqlens_write_nothing(gpu_lib):
    g = torch.Generator().manual_seed(2)
    n, d = 40, 128
    q, k, v = (normal(g, n, 1, d).cuda() for _ in range(3))
    dims = gdn.make_attn_dims(1, 1, d)
    for cu_q, cu_kv in (([0, 30, 20, 40], None), ([1, 20, 30, 40], None), ([0, 20, 30, 41], None),
                        ([0, 20, 30, 39], None), ([0, 20, 30, 40], [0, 20, 50, 40]),
                        ([0, -5, 30, 40], None)):
        o = torch.full((n, 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_attn_prefill(dims, q, k, v, _ints(cu_q), None if cu_kv is None else _ints(cu_kv),
                             o=o, d_status=status)
        assert status.item() == gdn.GDN_DEV_BAD_CU_SEQLENS, cu_q
        assert (o == 7).all()


def test_many_sequences(gpu_lib):
    """More sequences than a CTA has threads: the search for a block's sequence
    takes several turns."""
    g = torch.Generator().manual_seed(6)
    lens = [(i * 7) % 5 for i in range(700)]
    cu, hq, hkv, d = _cu(lens), 2, 1, 64
    q, k, v = (normal(g, cu[-1], h, d) for h in (hq, hkv, hkv))
    o = _run(gdn.make_attn_dims(hq, hkv, d), q.cuda(), k.cuda(), v.cuda(), cu)
    ref, slack = _attn.prefill(q, k, v, cu, cu, None, _attn.scale_of(d), torch.bfloat16)
    _attn.check(o, ref, slack, torch.bfloat16, "o")


def test_large_batch_matches_a_float32_form_and_repeats_bit_for_bit(gpu_lib):
    """More row blocks than SMs: against a plain fp32 form on the GPU, by the
    2-norm (rounding of weights and outputs: two half steps and margin)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n, hq, hkv, d = 3001, 16, 4, 256
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").to(torch.bfloat16)
               for h in (hq, hkv, hkv))
    dims = gdn.make_attn_dims(hq, hkv, d)
    cu = [0, 1200, 1201, 3001]
    o = _run(dims, q, k, v, cu)
    assert torch.equal(o, _run(dims, q, k, v, cu))
    ref = torch.empty(n, hq, d, device="cuda")
    for a, b in zip(cu, cu[1:]):
        kk, vv = (x[a:b].float().repeat_interleave(hq // hkv, 1).transpose(0, 1) for x in (k, v))
        s = q[a:b].float().transpose(0, 1) @ kk.transpose(1, 2) / 16
        s.masked_fill_(torch.ones(b - a, b - a, device="cuda").triu(1).bool(), -float("inf"))
        ref[a:b] = (torch.softmax(s, -1) @ vv).transpose(0, 1)
    assert float((o.float() - ref).norm() / ref.norm()) < 2 * 2.0 ** -8


def test_on_another_stream_and_from_a_graph(gpu_lib):
    g = torch.Generator().manual_seed(5)
    n, hq, hkv, d = 333, 4, 2, 256
    q, k, v = (normal(g, n, h, d).cuda() for h in (hq, hkv, hkv))
    dims, cu = gdn.make_attn_dims(hq, hkv, d), _ints([0, 100, n])
    plain = gdn.gdn_attn_prefill(dims, q, k, v, cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o = gdn.gdn_attn_prefill(dims, q, k, v, cu)
    side.synchronize()
    assert torch.equal(o, plain)
    o = torch.zeros_like(plain)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        gdn.gdn_attn_prefill(dims, q, k, v, cu, o=o)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, plain)


def test_an_output_on_a_16_byte_boundary(gpu_lib):
    g = torch.Generator().manual_seed(25)
    n, d = 130, 128
    q, k, v = (normal(g, n, 2, d).cuda() for _ in range(3))
    dims, cu = gdn.make_attn_dims(2, 2, d), _ints([0, n])
    plain = gdn.gdn_attn_prefill(dims, q, k, v, cu)
    room = torch.zeros(n * 2 * d + 8, dtype=torch.bfloat16, device="cuda")
    o = room[8:].view(n, 2, d)
    assert o.data_ptr() % 32 == 16
    gdn.gdn_attn_prefill(dims, q, k, v, cu, o=o)
    assert torch.equal(o, plain) and (room[:8] == 0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_sequence_alone_and_in_a_batch_gives_the_same_bits(gpu_lib, d):
    """Rows that share a warp with another sequence's, or with none, round alike."""
    g = torch.Generator().manual_seed(26)
    lens, hq, hkv = [37, 461, 90], 4, 2
    cu = _cu(lens)
    q, v = normal(g, cu[-1], hq, d).cuda(), normal(g, cu[-1], hkv, d).cuda()
    k = (3 * normal(g, cu[-1], hkv, d)).cuda()
    dims = gdn.make_attn_dims(hq, hkv, d)
    o = _run(dims, q, k, v, cu)
    for a, b in zip(cu, cu[1:]):
        assert torch.equal(o[a:b], _run(dims, q[a:b], k[a:b], v[a:b], [0, b - a]))


@pytest.mark.parametrize("d,hq,hkv,io,gate", [(64, 6, 6, "bf16", True), (64, 8, 4, "fp16", False),
                                              (128, 8, 4, "bf16", True), (128, 12, 4, "fp16", False),
                                              (256, 4, 4, "bf16", True)])
def test_many_short_items_follow_each_other(gpu_lib, d, hq, hkv, io, gate):
    """Far more row blocks than the GPU runs at a time, of one key block, of
    several and of none, so that each stage works on another item."""
    g = torch.Generator().manual_seed(d + hq)
    lens_q = [(37 * i) % 97 if i % 7 else 0 for i in range(400)]
    lens_kv = [n if i % 3 else (0, 1, n + 130, n // 2)[i // 3 % 4] for i, n in enumerate(lens_q)]
    cu_q, cu_kv, dt = _cu(lens_q), _cu(lens_kv), IO[io]
    qg, kv = normal(g, cu_q[-1], hq, 2 * d, dtype=dt), normal(g, cu_kv[-1], 2 * hkv, d, dtype=dt)
    qgd, kvd = qg.cuda(), kv.cuda()
    o = _run(gdn.make_attn_dims(hq, hkv, d, io=io), qgd[..., :d], kvd[:, :hkv], kvd[:, hkv:], cu_q,
             cu_kv, qgd[..., d:] if gate else None)
    ref, slack = _attn.prefill(qg[..., :d], kv[:, :hkv], kv[:, hkv:], cu_q, cu_kv,
                               qg[..., d:] if gate else None, _attn.scale_of(d), dt)
    _attn.check(o, ref, slack, dt, "o")
