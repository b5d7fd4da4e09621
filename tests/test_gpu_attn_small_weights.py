"""Softmax weights far below the largest: many keys of a weight near 2^-25 of
one key's come to something together.  In fp16, where such a weight lies below
the type's smallest step unless it is scaled, they must not be lost.

One key has score 0 and value 0; all others have a score of -18 (in units of
ln: their weight is exp(-18) = 2^-25.97) and value 2048.  With n of them
  o = 2048 n w / (1 + n w),  w = exp(-18),
which is 0.064 for n = 2047.  Every weight may be off by its own rounding
(half a step, relative) and by what fp32 leaves: the bound is the one of
tests/_attn.py."""
import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _attn
from tests._attn import IO

pytestmark = pytest.mark.gpu


def _inputs(n, first, d, dt):
    """q, k, v [n, 1, d]: key `first` scores 0, the others -18 at scale 1."""
    q, k, v = (torch.zeros(n, 1, d, dtype=dt) for _ in range(3))
    q[..., 0] = 1
    k[..., 0] = -18
    v[...] = 2048
    k[first], v[first] = 0, 0
    return q, k, v


@pytest.mark.parametrize("io", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("first", [0, 1000])
def test_prefill(gpu_lib, io, d, first):
    dt, n = IO[io], 2048
    q, k, v = _inputs(n, first, d, dt)
    q = q[-3:]
    dims = gdn.make_attn_dims(1, 1, d, io=io, scale=1.0)
    cu, cu_kv = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in ([0, 3], [0, n]))
    o = gdn.gdn_attn_prefill(dims, q.cuda(), k.cuda(), v.cuda(), cu, cu_kv)
    ref, slack = _attn.prefill(q, k, v, [0, 3], [0, n], None, 1.0, dt)
    _attn.check(o, ref, slack, dt, "o")


@pytest.mark.parametrize("io", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("shared", [0, 1024])
@pytest.mark.parametrize("width", [2048, 16384])
def test_decode(gpu_lib, io, d, shared, width):
    dt, n, page, rows = IO[io], 2048, 64, 2
    q, k, v = _inputs(n, 1000, d, dt)
    q = q[:rows]
    kc, vc = (x.view(n // page, page, 1, d).transpose(1, 2).contiguous() for x in (k, v))
    table = torch.full((rows, width // page), -1, dtype=torch.int32)
    table[:, :n // page] = torch.arange(n // page)
    dims = gdn.make_attn_dims(1, 1, d, io=io, page_size=page, scale=1.0)
    ws = torch.empty(gdn.gdn_attn_decode_workspace_size(dims, rows, shared), dtype=torch.uint8,
                     device="cuda")
    lens = [n, n - 50]
    o = gdn.gdn_attn_decode(dims, q.cuda(), kc.cuda(), vc.cuda(), table.cuda(),
                            torch.tensor(lens, dtype=torch.int32, device="cuda"), ws,
                            shared_len=shared)
    ref, slack = _attn.decode(q, kc, vc, table, lens, None, 1.0, dt)
    _attn.check(o, ref, slack, dt, "o")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_weights_stay_in_range(gpu_lib, d):
    """The reference maximum may lag behind the true one (by up to 2^8): scores
    that creep up by less than that from block to block, in fp16, with values
    near the type's largest.  Weights and their products must not overflow."""
    n, dt = 1024, torch.float16
    q, k, v = (torch.zeros(n, 1, d, dtype=dt) for _ in range(3))
    q[..., 0] = 1
    k[..., 0] = torch.linspace(0, 16, n)[:, None]
    v[...] = 60000.0 * torch.where(torch.arange(n) % 3 == 0, -1.0, 1.0)[:, None, None]
    q = q[-5:]
    dims = gdn.make_attn_dims(1, 1, d, io="fp16", scale=1.0)
    cu, cu_kv = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in ([0, 5], [0, n]))
    o = gdn.gdn_attn_prefill(dims, q.cuda(), k.cuda(), v.cuda(), cu, cu_kv)
    ref, slack = _attn.prefill(q, k, v, [0, 5], [0, n], None, 1.0, dt)
    _attn.check(o, ref, slack, dt, "o")
