"""Axes that no pair turns by: a model's positions have a row for each of its axes, also where the
last section of its pairs is empty."""
import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests.test_attn_marshalling import D, HKV, HQ, N, Tensor, _ints
from tests.test_attn_marshalling import calls as attn_calls  # noqa: F401
from tests.test_kv8_marshalling import _cache, calls  # noqa: F401


def test_the_number_of_axes():
    assert gdn.make_rope_axes([0, 0, 1]).count == 2
    a = gdn.make_rope_axes([0, 0, 1], count=3)
    assert a.count == 3 and list(a.pair[:3]) == [0, 0, 1]
    assert gdn.make_rope_axes([], count=4).count == 4
    assert gdn.make_rope_axes([0, 1], count=2).count == 2
    for axis, count in (([0, 1], 1), ([0], 0), ([0], -1), ([0], 5), ([0, 3], 3)):
        with pytest.raises(ValueError):
            gdn.make_rope_axes(axis, count=count)


@pytest.mark.parametrize("sections", [[24, 8, 0], [32, 0, 0], [16, 0, 16]])
def test_positions_of_every_axis_are_taken(calls, sections):  # noqa: F811
    axes = gdn.make_rope_axes(gdn.rope_sections(sections), count=len(sections))
    q, k, v = (Tensor((N, h, D)) for h in (HQ, HKV, HKV))
    dims, pos = gdn.make_attn_dims(HQ, HKV, D, page_size=16), _ints(3, N)
    gdn.gdn_qk_norm_rope_axes(dims, q, k, None, None, None, pos, axes)
    assert calls.args[6] == N and calls.axes.count == 3
    gdn.gdn_kv8_append(dims, q, k, v, None, None, None, pos, _cache(), _ints(N), axes=axes)
    assert calls.args[10] == N


def test_positions_of_other_axes_are_refused_by_their_name(calls):  # noqa: F811
    q, k, v = (Tensor((N, h, D)) for h in (HQ, HKV, HKV))
    dims, pos = gdn.make_attn_dims(HQ, HKV, D, page_size=16), _ints(3, N)
    for axes in (gdn.make_rope_axes([0, 1]), gdn.make_rope_axes([0, 1], count=4)):
        with pytest.raises(ValueError, match="positions has 9 elements"):
            gdn.gdn_qk_norm_rope_axes(dims, q, k, None, None, None, pos, axes)
        with pytest.raises(ValueError, match="positions has 9 elements"):
            gdn.gdn_qk_norm_rope_axes(dims, None, k, None, None, None, pos, axes)
        with pytest.raises(ValueError, match="positions has 9 elements"):
            gdn.gdn_kv8_append(dims, q, k, v, None, None, None, pos, _cache(), _ints(N), axes=axes)


@pytest.mark.gpu
@pytest.mark.parametrize("sections", [[24, 8, 0], [32, 0, 0], [0, 32, 0]])
@pytest.mark.parametrize("n", [5, 700])
def test_an_empty_section_turns_nothing(gpu_lib, n, sections):
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, 2, 128, generator=g).bfloat16().cuda()
    pos = torch.randint(0, 9000, (3, n), generator=g, dtype=torch.int32).cuda()
    freq = gdn.rope_frequencies(64, 1e6, device="cuda")[0]
    dims = gdn.make_attn_dims(2, 2, 128, rot_dim=64, page_size=16)
    axis = gdn.rope_sections(sections)
    axes = gdn.make_rope_axes(axis, count=3)
    q, _ = gdn.gdn_qk_norm_rope_axes(dims, x, None, None, None, freq, pos, axes)
    used = max(axis) + 1
    plain, _ = gdn.gdn_qk_norm_rope_axes(dims, x, None, None, None, freq, pos[:used].contiguous(),
                                         gdn.make_rope_axes(axis))
    width = -(-n // 16)
    cache = gdn.make_kv8_cache(dims, width, torch.arange(width, dtype=torch.int32, device="cuda").view(1, -1))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    k_out = torch.empty_like(x)
    o = gdn.gdn_kv8_append(dims, x, x, x, None, None, freq, pos, cache, cu[:1], cu_seqlens=cu, axes=axes,
                           k_out=k_out)
    torch.cuda.synchronize()
    assert torch.equal(q, plain) and torch.equal(o, plain) and torch.equal(k_out, plain)
