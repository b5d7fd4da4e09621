"""Attention calls sent to another stream by their `stream` argument, outputs
not given: the output is memory of that stream.  Were it a block of the current
stream's that has just been freed, what that stream still has to do with it
would land in the output after the call."""
import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests._attn import normal

pytestmark = pytest.mark.gpu
N, HQ, HKV, D, PAGE = 640, 4, 2, 128, 64


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _calls():
    g = torch.Generator().manual_seed(3)
    q, k, v = (normal(g, N, h, D).cuda() for h in (HQ, HKV, HKV))
    pos, w = torch.arange(N, dtype=torch.int32, device="cuda"), torch.ones(D, device="cuda")
    freq = gdn.rope_frequencies(64, 1e6, device="cuda")[0]
    dims = gdn.make_attn_dims(HQ, HKV, D, rot_dim=64, page_size=PAGE)
    kc, vc = (normal(g, N, HKV, PAGE, D).cuda() for _ in range(2))
    table, lens = pos.view(N, 1), torch.full((N,), PAGE, dtype=torch.int32, device="cuda")
    ws = torch.empty(gdn.gdn_attn_decode_workspace_size(dims, N), dtype=torch.uint8, device="cuda")
    cu, zeros = _ints([0, 300, N]), torch.zeros(N, dtype=torch.int32, device="cuda")
    kc2, vc2 = kc.clone(), vc.clone()
    return {"norm_rope": lambda **s: gdn.gdn_qk_norm_rope(dims, q, k, w, w, freq, pos, **s)[0],
            "append": lambda **s: gdn.gdn_kv_append(dims, q, k, v, w, w, freq, zeros, kc2, vc2, table,
                                                    **s),
            "prefill": lambda **s: gdn.gdn_attn_prefill(dims, q, k, v, cu, **s),
            "decode": lambda **s: gdn.gdn_attn_decode(dims, q, kc, vc, table, lens, ws, **s)}


@pytest.mark.parametrize("name", ["norm_rope", "append", "prefill", "decode"])
def test_work_that_the_current_stream_still_has_to_do_stays_out(gpu_lib, name):
    call = _calls()[name]
    plain = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # a block of the output's size, freed with a write to it still to come
    was = torch.empty_like(plain)
    torch.cuda._sleep(100_000_000)
    was.fill_(7.0)
    del was
    o = call(stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(o, plain)
    spans = [(s["address"], s["address"] + s["total_size"], s["stream"])
             for s in torch.cuda.memory_snapshot()]
    assert [s for a, b, s in spans if a <= o.data_ptr() < b] == [side.cuda_stream]


def test_the_default_stream_by_its_handle(gpu_lib):
    call = _calls()["prefill"]
    plain = call()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        o = call(stream=0)
    torch.cuda.synchronize()
    assert torch.equal(o, plain)
