"""gdn_attn_decode behind a shared prefix that some rows end inside of: such a
row sees its own first tokens of the prefix and nothing of what lies after
them there, whatever that is."""
import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _attn
from tests._attn import IO, normal

pytestmark = pytest.mark.gpu


def _prefix_tail(cache, pages, page, start, shared, bad):
    """Tokens [start, shared) of the prefix's pages set to `bad`."""
    for t in range(start, shared):
        cache[int(pages[t // page]), :, t % page] = bad


CASES = [   # lengths, hq, hkv, d, page, io, gate, shared, the first token that is bad
    ([100, 37, 1, 0, 65], 4, 2, 256, 64, "bf16", True, 640, 100),
    ([200, 129], 6, 2, 128, 16, "fp16", False, 272, 200),
    ([3, 2], 4, 4, 64, 32, "bf16", False, 96, 3),
    ([63, 64, 65, 127, 128], 40, 2, 128, 128, "bf16", True, 256, 128),
    ([250] * 70, 4, 2, 64, 64, "fp16", True, 320, 250),         # two row blocks of the prefix
    ([5000, 130, 7000], 16, 4, 256, 64, "bf16", True, 8192, 7000),
    ([900, 40], 16, 1, 64, 16, "bf16", True, 4096, 900),
]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens,hq,hkv,d,page,io,gate,shared,start", CASES)
def test_rows_that_end_inside_the_prefix(gpu_lib, lens, hq, hkv, d, page, io, gate, shared, start,
                                         bad):
    g = torch.Generator().manual_seed(sum(lens) + d)
    dt, n = IO[io], len(lens)
    # a cache for sequences of the prefix's length, the prefix then bad from `start` on
    kc, vc, table = _attn.paged(g, [shared] * n, hkv, d, page, dt, shared=shared)
    for c in (kc, vc):
        _prefix_tail(c, table[0], page, start, shared, bad)
    table[1:, :shared // page] = -1          # only the first row's entries are looked at there
    qg = normal(g, n, hq, 2 * d, dtype=dt)
    dims = gdn.make_attn_dims(hq, hkv, d, io=io, page_size=page)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((gdn.gdn_attn_decode_workspace_size(dims, n, shared),), 0xff, dtype=torch.uint8,
                    device="cuda")
    qgd = qg.cuda()
    o = gdn.gdn_attn_decode(dims, qgd[..., :d], kc.cuda(), vc.cuda(), table.cuda(),
                            torch.tensor(lens, dtype=torch.int32, device="cuda"), ws,
                            shared_len=shared, gate=qgd[..., d:] if gate else None, d_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    ref, slack = _attn.decode(qg[..., :d], kc, vc, table[:1].expand(n, -1), lens,
                              qg[..., d:] if gate else None, _attn.scale_of(d), dt)
    _attn.check(o, ref, slack, dt, "o")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_short_rows_beside_long_ones(gpu_lib, d):
    """Rows on both sides of the prefix's end, all finite: each as without the
    prefix, and the rows behind it not touched by what a short row's own pages
    hold."""
    g = torch.Generator().manual_seed(d)
    lens, hq, hkv, page, shared = [1500, 300, 512, 511, 0, 513, 1], 8, 2, 32, 512
    n = len(lens)
    kc, vc, table = _attn.paged(g, lens, hkv, d, page, torch.bfloat16, shared=shared)
    q = normal(g, n, hq, d)
    dims = gdn.make_attn_dims(hq, hkv, d, page_size=page)
    ws = torch.full((gdn.gdn_attn_decode_workspace_size(dims, n, shared),), 0xff, dtype=torch.uint8,
                    device="cuda")
    o = gdn.gdn_attn_decode(dims, q.cuda(), kc.cuda(), vc.cuda(), table.cuda(),
                            torch.tensor(lens, dtype=torch.int32, device="cuda"), ws,
                            shared_len=shared)
    ref, slack = _attn.decode(q, kc, vc, table, lens, None, _attn.scale_of(d), torch.bfloat16)
    _attn.check(o, ref, slack, torch.bfloat16, "o")
