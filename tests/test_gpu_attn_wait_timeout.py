"""The bounded waits of the full-attention kernels, made to run out.

With GDN_TEST_WAIT_TIMEOUT (a test-only flag of gdn_attn_dims) the waits give up
after 2 ms instead of 4 s and some hand-overs inside the kernels never come:
whoever waits for them must give up, report GDN_DEV_WAIT_TIMEOUT and end, the
other work of the call unharmed, the next call on the stream as if nothing had
been.  Nothing here faults, traps or waits without a bound."""
import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _attn
from tests._attn import normal

pytestmark = pytest.mark.gpu


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _rows_right_or_untouched(o, ref, slack, what):
    """Every row of o is right, or still the 7.0 it was filled with; returns how many are not."""
    o = o.cpu()
    out = (o == 7).all(-1)
    rows = ~out
    _attn.check(o[rows], ref[rows], slack[rows], o.dtype, what)
    return int(out.sum())


# Items of one key block whose values end inside it, of whole blocks, of several with an
# end; pairs (heads of 128 and 256) and single CTAs, with more items than are under way.
@pytest.mark.parametrize("lens,hq,hkv,d,gate", [
    ([40], 4, 2, 256, True), ([40, 50, 60], 2, 1, 128, False), ([40] * 5, 2, 2, 64, True),
    ([512], 2, 2, 256, False), ([512, 256], 2, 1, 128, True), ([512], 2, 2, 64, False),
    ([700, 1000, 30], 4, 2, 256, True), ([700, 1000, 30], 4, 2, 128, False),
    ([700, 1000, 30], 4, 2, 64, False), ([150] * 130, 4, 4, 128, False), ([150] * 90, 4, 4, 256, False),
    ([150] * 130, 4, 4, 64, True),
])
def test_prefill(gpu_lib, lens, hq, hkv, d, gate):
    g = torch.Generator().manual_seed(sum(lens) + d)
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    qg, k, v = normal(g, cu[-1], hq, 2 * d), normal(g, cu[-1], hkv, d), normal(g, cu[-1], hkv, d)
    ref, slack = _attn.prefill(qg[..., :d], k, v, cu, cu, qg[..., d:] if gate else None,
                               _attn.scale_of(d), torch.bfloat16)
    qgd, kd, vd = qg.cuda(), k.cuda(), v.cuda()

    def call(flags):
        o = torch.full((cu[-1], hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        status = _status()
        gdn.gdn_attn_prefill(gdn.make_attn_dims(hq, hkv, d, flags=flags), qgd[..., :d], kd, vd,
                             _ints(cu), gate=qgd[..., d:] if gate else None, o=o, d_status=status)
        torch.cuda.synchronize()
        return o, status.item()
    o, status = call(gdn.GDN_TEST_WAIT_TIMEOUT)
    assert status == gdn.GDN_DEV_WAIT_TIMEOUT
    assert _rows_right_or_untouched(o, ref, slack, "with waits that ran out") > 0
    o, status = call(0)
    assert status == 0
    _attn.check(o, ref, slack, torch.bfloat16, "the next call")


# The form for few keys (a cluster per row), runs of units with a merge, and both passes behind
# a shared prefix.
@pytest.mark.parametrize("lens,hq,hkv,d,page,width,gate,shared", [
    ([700], 16, 4, 256, 64, 704, True, 0), ([300, 40], 4, 2, 128, 16, 320, False, 0),
    ([500, 20], 8, 8, 64, 32, 512, True, 0), ([3000] * 8, 4, 2, 256, 64, 8192, True, 0),
    ([6000] * 3, 4, 2, 128, 64, 8192, False, 0), ([2500] * 20, 4, 4, 64, 128, 4096, True, 0),
    ([3000, 2500, 2100], 8, 2, 256, 64, 4096, True, 2048),
    ([600, 513], 4, 2, 128, 16, 1024, False, 512), ([2100] * 40, 4, 2, 64, 64, 4096, False, 2048),
])
def test_decode(gpu_lib, lens, hq, hkv, d, page, width, gate, shared):
    g = torch.Generator().manual_seed(sum(lens) + d)
    n = len(lens)
    kc, vc, table = _attn.paged(g, lens, hkv, d, page, torch.bfloat16, shared=shared)
    wide = torch.full((n, width // page), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    qg = normal(g, n, hq, 2 * d)
    ref, slack = _attn.decode(qg[..., :d], kc, vc, table, lens, qg[..., d:] if gate else None,
                              _attn.scale_of(d), torch.bfloat16)
    qgd, kcd, vcd, wide, ln = qg.cuda(), kc.cuda(), vc.cuda(), wide.cuda(), _ints(lens)
    ws = torch.zeros(gdn.gdn_attn_decode_workspace_size(
        gdn.make_attn_dims(hq, hkv, d, page_size=page), n, shared), dtype=torch.uint8, device="cuda")

    def call(flags):
        status = _status()
        o = gdn.gdn_attn_decode(gdn.make_attn_dims(hq, hkv, d, page_size=page, flags=flags),
                                qgd[..., :d], kcd, vcd, wide, ln, ws, shared_len=shared,
                                gate=qgd[..., d:] if gate else None, d_status=status)
        torch.cuda.synchronize()
        return o, status.item()
    o, status = call(gdn.GDN_TEST_WAIT_TIMEOUT)
    assert status == gdn.GDN_DEV_WAIT_TIMEOUT
    if not shared:      # rows are right, or seen to be not valid
        o, bad = o.cpu(), torch.isnan(o.cpu()).any(-1)
        assert bad.any()
        _attn.check(o[~bad], ref[~bad], slack[~bad], torch.bfloat16, "with waits that ran out")
    o, status = call(0)
    assert status == 0
    _attn.check(o, ref, slack, torch.bfloat16, "the next call")


@pytest.mark.parametrize("n,hq,hkv,d,io,layout", [
    (700, 16, 4, 256, "bf16", "half"), (3001, 16, 4, 128, "fp16", "interleaved"),
    (1000, 40, 8, 256, "bf16", "half"), (2000, 4, 4, 64, "fp32", "interleaved"),
])
def test_norm_and_rotation(gpu_lib, n, hq, hkv, d, io, layout):
    g = torch.Generator().manual_seed(n)
    dt = _attn.IO[io]
    q, k, w = normal(g, n, hq, d, dtype=dt), normal(g, n, hkv, d, dtype=dt), 1 + 0.1 * torch.randn(d, generator=g)
    pos, freq = torch.arange(n, dtype=torch.int32), gdn.rope_frequencies(d // 2, 1e6)[0]
    refs = [_attn.norm_rope(x, w, 1e-6, pos, freq, layout) for x in (q, k)]
    qd, kd, wd, posd, freqd = q.cuda(), k.cuda(), w.cuda(), pos.cuda(), freq.cuda()
    page = 16
    table = torch.arange(-(-n // page), dtype=torch.int32, device="cuda")[None]
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")

    def call(flags, append):
        dims = gdn.make_attn_dims(hq, hkv, d, io=io, rot_dim=d // 2, rope=layout, page_size=page,
                                  flags=flags)
        status = _status()
        qo, ko = (torch.full(x.shape, 7.0, dtype=dt, device="cuda") for x in (q, k))
        if append:
            kc = torch.full((table.shape[1], hkv, page, d), 7.0, dtype=dt, device="cuda")
            vc = kc.clone()
            gdn.gdn_kv_append(dims, qd, kd, kd, wd, wd, freqd, posd, kc, vc, table, row_seq=seq,
                              q_out=qo, d_status=status)
            ko, vo = (c.transpose(1, 2).reshape(-1, hkv, d)[:n] for c in (kc, vc))
        else:
            gdn.gdn_qk_norm_rope(dims, qd, kd, wd, wd, freqd, posd, qo, ko, d_status=status)
            vo = None
        torch.cuda.synchronize()
        return (qo, ko, vo), status.item()
    for append in (False, True):
        outs, status = call(gdn.GDN_TEST_WAIT_TIMEOUT, append)
        assert status == gdn.GDN_DEV_WAIT_TIMEOUT
        for o, (ref, slack) in zip(outs, refs):
            assert _rows_right_or_untouched(o, ref, slack, "with waits that ran out") > 0
        outs, status = call(0, append)
        assert status == 0
        for o, (ref, slack) in zip(outs, refs):
            _attn.check(o, ref, slack, dt, "the next call")
        if append:
            assert torch.equal(outs[2].cpu(), k)
