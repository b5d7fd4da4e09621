"""The example that runs the full-attention layer's calls together: its last
step against a plain fp32 attention over what the cache then holds, by the
2-norm (the rounding of weights and outputs: two half steps)."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests,common,own,steps", [(5, 256, 37, 3), (1, 128, 1, 2), (3, 0, 70, 2)])
def test_layer_over_a_common_prompt(gpu_lib, requests, common, own, steps):
    import full_attention_layer as example
    r = example.run(requests, common, own, steps)
    ref = example.plain(r)
    assert int(r["lens"][0]) == common + own + steps
    assert float((r["o"].float() - ref).norm() / ref.norm()) < 2 * 2.0 ** -8
