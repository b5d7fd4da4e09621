"""The example that serves from the 8-bit cache: its last step against a plain fp32 attention
over the cache's numbers, by the 2-norm (the rounding of weights and outputs: two half
steps), and what the cached tokens received: a step gives 1 per query head, and an eviction
keeps no more than there was."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests,text,side,steps,keep,evictions",
                         [(5, 20, 6, 4, 50, 3), (2, 3, 2, 2, 100, 0), (3, 40, 5, 30, 64, 2)])
def test_requests_with_images(gpu_lib, requests, text, side, steps, keep, evictions):
    import eight_bit_cache as example
    import gated_deltanet_linear_07_gb300 as gdn
    assert example.H_Q % example.H_KV == 0 and gdn.GDN_KV8_BLOCK == 16
    r = example.run(requests, text, side, steps, keep)
    ref = example.plain(r)
    assert r["evictions"] == evictions and r["prompt"] == 2 * text + side * side
    assert float((r["o"].float() - ref).norm() / ref.norm()) < 2 * 2.0 ** -8
    w = r["weights"].double()
    assert (w >= 0).all() and not w[:, :, r["length"]:].any()
    most = steps * (example.H_Q // example.H_KV)
    assert (w.sum(-1) <= most * (1 + 2.0 ** -16)).all()
