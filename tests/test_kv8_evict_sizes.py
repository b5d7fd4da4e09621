"""Evictions of more sequences, heads and kept places than their launches can have CTAs are refused
before the first launch (fake addresses, on a host without a GPU: nothing below is launched)."""
import pytest

import gated_deltanet_linear_07_gb300 as gdn
from tests.test_attn_refusals import A
from tests.test_kv8_refusals import cache, evict, lib  # noqa: F401

MOST = (1 << 31) - 1
PAGE = gdn.make_attn_dims(**A).page_size
LONG = ((1 << 31) - (1 << 16)) // PAGE        # pages of the longest block table row


@pytest.mark.parametrize("h,n,keep", [
    (2, 1 << 30, 1),                          # a head of a sequence more than the selection's CTAs
    (65535, MOST, 1),
    (65535, MOST, LONG * PAGE),               # their product past 64 bits
    (4, 1 << 20, 1 << 24),                    # the selection's fit, the copy's do not
    (1, 257, LONG * PAGE),                    # 2^8 + 1 sequences of 2^23 - 2^8 CTAs (2^8 fit), and
    (1, 1 << 30, 16 * 16 * 2 + 1),            # 2^30 of 3
])
def test_more_ctas_than_a_launch_takes(lib, h, n, keep):  # noqa: F811
    dims = gdn.make_attn_dims(**dict(A, h_q=h, h_kv=h))
    from_, to = cache(pages=1, seqs=MOST), cache(pages=1, seqs=MOST, per=LONG)
    assert evict(lib, dims, c=from_, to=to, n=n, keep=keep) == -2
