"""gdn_attn_prefill with values that are no numbers: how far they reach.

Masked weights are zeros, and zero times NaN or Inf is NaN: a block of query
rows (256 tokens at most) multiplies every block of 128 keys up to the last one
that its last token sees.  So a value at key s can reach queries up to
256 - 1 + 128 - 1 = 382 tokens before it, and no others before it."""
import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _attn
from tests._attn import normal

pytestmark = pytest.mark.gpu
REACH = 382


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (2, 2, 128), (3, 1, 128), (1, 1, 256), (4, 1, 256)])
@pytest.mark.parametrize("n,before,at", [(700, 0, 200), (900, 0, 899), (900, 77, 800), (500, 300, 640),
                                         (383, 0, 382), (384, 0, 383)])
def test_reach_of_a_value(gpu_lib, hq, hkv, d, n, before, at, bad):
    g = torch.Generator().manual_seed(n + d)
    q, k, v = normal(g, n, hq, d), normal(g, n + before, hkv, d), normal(g, n + before, hkv, d)
    v[at] = bad
    cu, cu_kv = (torch.tensor([0, x], dtype=torch.int32, device="cuda") for x in (n, n + before))
    o = gdn.gdn_attn_prefill(gdn.make_attn_dims(hq, hkv, d), q.cuda(), k.cuda(), v.cuda(), cu,
                             cu_kv).cpu()
    place = torch.arange(n) + before               # each query's own key
    assert not torch.isfinite(o[place >= at]).any()
    rest = place < at - REACH
    ref, slack = _attn.prefill(q[rest], k, v, [0, int(rest.sum())], [0, int(rest.sum()) + before],
                               None, _attn.scale_of(d), torch.bfloat16)
    _attn.check(o[rest], ref, slack, torch.bfloat16, "the rows before it")
