"""gdn_qk_norm_rope_axes against the 64-bit form: every pair turned by the position on its
own axis, few tokens and many (two kernels), every type, layout and head dim,
negative and far positions, several axes that agree, strided views."""
import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _attn
from tests._attn import E, IO, normal

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _reference(x, w, pos, axis, freq, layout, rope_scale):
    """_attn.norm_rope with the angle of pair i from pos[axis[i]]."""
    x = x.double()
    if w is not None:
        x = x / ((x * x).mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    y, size, half = x.clone(), x.abs(), freq.numel()
    for i in range(half):
        a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
        angle = pos[axis[i]].double() * freq[i]
        c, s = angle.cos()[:, None] * rope_scale, angle.sin()[:, None] * rope_scale
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
        size[..., a] = size[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(rope_scale)
    return y, 32 * E * size


CASES = [   # n, hq, hkv, d, rot, layout, io, axes, mixed
    (1, 16, 4, 256, 64, "half", "bf16", 3, True), (5, 4, 2, 64, 64, "interleaved", "fp16", 3, False),
    (130, 8, 8, 128, 128, "half", "fp32", 4, True), (639, 2, 1, 256, 32, "interleaved", "bf16", 2, False),
    (640, 2, 1, 128, 96, "half", "bf16", 3, True), (700, 3, 3, 64, 16, "half", "fp16", 4, False),
    (1027, 4, 1, 256, 256, "interleaved", "fp32", 3, True), (801, 2, 2, 128, 64, "half", "bf16", 1, False),
    (2500, 1, 1, 64, 64, "half", "bf16", 3, True),
]


@pytest.mark.parametrize("n,hq,hkv,d,rot,layout,io,axes,mixed", CASES)
def test_axes(gpu_lib, n, hq, hkv, d, rot, layout, io, axes, mixed):
    g = torch.Generator().manual_seed(n + d)
    dt = IO[io]
    pairs = rot // 2
    sections = [pairs // axes + (1 if a < pairs % axes else 0) for a in range(axes)]
    axis = gdn.rope_sections(sections, interleaved=mixed)
    assert len(axis) == pairs
    pos = torch.randint(-50, 300_000, (axes, n), generator=g, dtype=torch.int32)
    freq, scale = gdn.rope_frequencies(rot, 1e6)
    q, k = normal(g, n, hq, 2 * d, dtype=dt), normal(g, n, hkv + 1, d, dtype=dt)
    wq, wk = 1 + 0.1 * torch.randn(d, generator=g), 1 + 0.1 * torch.randn(d, generator=g)
    dims = gdn.make_attn_dims(hq, hkv, d, io=io, rot_dim=rot, rope=layout, norm_eps=EPS)
    qd, kd = q.cuda()[..., d:], k.cuda()[:, 1:]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko = gdn.gdn_qk_norm_rope_axes(dims, qd, kd, wq.cuda(), wk.cuda(), freq.cuda(), pos.cuda(),
                                       gdn.make_rope_axes(axis), rope_scale=0.75, d_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for got, x, w, what in ((qo, q[..., d:], wq, "q"), (ko, k[:, 1:], wk, "k")):
        ref, slack = _reference(x, w, pos, axis, freq, layout, 0.75)
        _attn.check(got, ref, slack, dt, what)


@pytest.mark.parametrize("n", [3, 1000])
def test_axes_that_agree_are_one(gpu_lib, n):
    g = torch.Generator().manual_seed(n)
    q = normal(g, n, 4, 128).cuda()
    pos = torch.randint(0, 9000, (n,), generator=g, dtype=torch.int32).cuda()
    freq = gdn.rope_frequencies(64, 1e6, device="cuda")[0]
    dims = gdn.make_attn_dims(4, 4, 128, rot_dim=64)
    one, none = gdn.gdn_qk_norm_rope(dims, q, None, None, None, freq, pos)
    many, none2 = gdn.gdn_qk_norm_rope_axes(dims, q, None, None, None, freq,
                                            pos.expand(3, n).contiguous(),
                                            gdn.make_rope_axes([0, 1, 2, 0] * 8))
    torch.cuda.synchronize()
    assert none is None and none2 is None and torch.equal(one, many)


def test_in_place_and_in_a_graph(gpu_lib):
    g = torch.Generator().manual_seed(1)
    x = normal(g, 900, 4, 64).cuda()
    pos = torch.randint(0, 9000, (2, 900), generator=g, dtype=torch.int32).cuda()
    freq = gdn.rope_frequencies(64, 1e4, device="cuda")[0]
    dims = gdn.make_attn_dims(4, 4, 64, rot_dim=64)
    axes = gdn.make_rope_axes(gdn.rope_sections([16, 16]))
    ref = gdn.gdn_qk_norm_rope_axes(dims, x, None, None, None, freq, pos, axes)[0]
    y = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_qk_norm_rope_axes(dims, y, None, None, None, freq, pos, axes, q_out=y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ref)
