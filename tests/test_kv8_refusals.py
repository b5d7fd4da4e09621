"""Positions with several axes, the 8-bit cache and eviction: what the entry points refuse, on a
host without a GPU (every call below fails validation or has nothing to do, and never
reaches the CUDA runtime), the workspace's size, the sections of axes, and the
binding's checks of its tensors."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from gated_deltanet_linear_07_gb300 import _binding
from tests.test_attn_refusals import BAD_DIMS, FAKE, A, view

BAD16 = BAD_DIMS + [(dict(A, io="fp32"), -2)]
BAD_PAGES = [(dict(A, page_size=48), -2), (dict(A, page_size=256), -2), (dict(A, page_size=8), -2)]


@pytest.fixture(scope="module")
def lib():
    gdn.build()
    return gdn.load()


def axes(count=3, pair=None):
    return gdn.gdn_rope_axes(count, (ctypes.c_uint8 * 128)(*(pair or [0, 1, 2] * 10 + [0, 0])))


def norm_rope(lib, dims=None, ax=axes(), q=view(), k=view(hs=256), pos=FAKE, n=4, q_out=FAKE,
              k_out=FAKE):
    p = gdn.gdn_rope_params(FAKE, FAKE, FAKE, 1.0)
    d = dims or gdn.make_attn_dims(**A)
    return lib.gdn_qk_norm_rope_axes(ctypes.byref(d), ctypes.byref(p), _binding._ref(ax),
                                     _binding._ref(q), _binding._ref(k), pos, n, q_out, k_out, None)


def test_axes_refusals(lib):
    for kw, rc in BAD_DIMS:
        assert norm_rope(lib, gdn.make_attn_dims(**kw)) == rc, kw
    assert norm_rope(lib, ax=None) == -1
    assert norm_rope(lib, ax=axes(0)) == -1
    assert norm_rope(lib, ax=axes(-1)) == -1
    assert norm_rope(lib, ax=axes(5)) == -1
    assert norm_rope(lib, ax=axes(2)) == -1                       # a pair on the third of two
    assert norm_rope(lib, ax=axes(1, [0] * 31 + [1])) == -1
    assert norm_rope(lib, ax=axes(1, [0] * 32 + [9]), n=0) == 0    # beyond the rotated pairs
    assert norm_rope(lib, n=0) == 0
    assert norm_rope(lib, n=-1) == -1
    assert norm_rope(lib, q=None, k=None) == -1
    assert norm_rope(lib, pos=None) == -1
    assert norm_rope(lib, q_out=None) == -1
    assert norm_rope(lib, k_out=FAKE + 8) == -5
    assert norm_rope(lib, q=view(hs=0)) == -2


def cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, table=FAKE, pages=100, seqs=8, per=10):
    return gdn.gdn_kv8_cache(k, v, ks, vs, table, pages, seqs, per)


BAD_CACHES = [(dict(k=None), -1), (dict(v=None), -1), (dict(ks=None), -1), (dict(vs=None), -1),
              (dict(table=None), -1), (dict(pages=0), -1), (dict(seqs=-1), -1), (dict(per=0), -1),
              (dict(k=FAKE + 8), -5), (dict(ks=FAKE + 2), -5), (dict(pages=1 << 31), -2),
              (dict(per=1 << 30), -2)]


def append(lib, dims=None, k=view(), v=view(), c=None, n=4, cu=FAKE, starts=FAKE, seqs=2, q_out=FAKE,
           q=view(), k_out=None, ax=None, pos=FAKE):
    p = gdn.gdn_rope_params(FAKE, FAKE, FAKE, 1.0)
    d = dims or gdn.make_attn_dims(**A)
    return lib.gdn_kv8_append(ctypes.byref(d), ctypes.byref(p), _binding._ref(ax), _binding._ref(q),
                              _binding._ref(k), _binding._ref(v), pos, cu, starts, seqs, n,
                              _binding._ref(c or cache()), q_out, k_out, None, None)


def test_append_refusals(lib):
    for kw, rc in BAD16 + BAD_PAGES:
        assert append(lib, gdn.make_attn_dims(**kw)) == rc, kw
    for kw, rc in BAD_CACHES:
        assert append(lib, c=cache(**kw)) == rc, kw
    assert append(lib, seqs=9) == -1                    # more sequences than the block table has
    assert append(lib, cu=None) == -1                   # two sequences for four rows of their own
    assert append(lib, cu=None, seqs=4, n=0) == -1
    assert append(lib, n=0) == 0
    assert append(lib, seqs=0) == -1
    assert append(lib, seqs=-1) == -1
    assert append(lib, n=-1) == -1
    assert append(lib, starts=None) == -1
    assert append(lib, pos=None) == -1
    assert append(lib, k=None) == -1
    assert append(lib, v=view(None)) == -1
    assert append(lib, q_out=None) == -1
    assert append(lib, ax=axes(2)) == -1
    assert append(lib, v=view(FAKE + 4)) == -5
    assert append(lib, k_out=FAKE + 8) == -5


def gather(lib, dims=None, c=None, cu=FAKE, seqs=2, total=4, k=FAKE, v=FAKE + 4096):
    d = dims or gdn.make_attn_dims(**A)
    return lib.gdn_kv8_gather(ctypes.byref(d), _binding._ref(c or cache()), cu, seqs, total, k, v, None,
                              None)


def test_gather_refusals(lib):
    for kw, rc in BAD16 + BAD_PAGES:
        assert gather(lib, gdn.make_attn_dims(**kw)) == rc, kw
    for kw, rc in BAD_CACHES:
        assert gather(lib, c=cache(**kw)) == rc, kw
    assert gather(lib, total=0) == 0
    assert gather(lib, total=-1) == -1
    assert gather(lib, total=1 << 31) == -2
    assert gather(lib, seqs=9) == -1
    assert gather(lib, seqs=0) == -1
    assert gather(lib, cu=None) == -1
    assert gather(lib, k=None, v=None) == -1
    assert gather(lib, v=FAKE) == -1                    # both into one
    assert gather(lib, k=FAKE + 4) == -5


def decode(lib, dims=None, q=view(), c=None, lens=FAKE, n=4, gate=None, weights=None, o=FAKE + 4096,
           ws=FAKE, size=1 << 40):
    d = dims or gdn.make_attn_dims(**A)
    return lib.gdn_attn_decode_kv8(ctypes.byref(d), _binding._ref(q), _binding._ref(c or cache()), lens,
                                   n, _binding._ref(gate), weights, o, ws, size, None, None)


def test_decode_refusals(lib):
    for kw, rc in BAD16 + BAD_PAGES:
        assert decode(lib, gdn.make_attn_dims(**kw)) == rc, kw
    for kw, rc in BAD_CACHES:
        assert decode(lib, c=cache(**kw)) == rc, kw
    assert decode(lib, n=0) == 0
    assert decode(lib, n=-1) == -1
    assert decode(lib, n=9) == -1
    assert decode(lib, q=None) == -1
    assert decode(lib, lens=None) == -1
    assert decode(lib, o=None) == -1
    assert decode(lib, o=FAKE) == -1                    # the output is an input
    assert decode(lib, gate=view(FAKE + 4096)) == -1
    assert decode(lib, o=FAKE + 4100) == -5
    assert decode(lib, weights=FAKE + 4) == -5
    assert decode(lib, ws=None) == -4
    assert decode(lib, ws=FAKE + 16) == -5
    d = gdn.make_attn_dims(**A)
    need = gdn.gdn_attn_decode_kv8_workspace_size(d, 4)
    more = gdn.gdn_attn_decode_kv8_workspace_size(d, 4, 640)
    assert decode(lib, size=need - 1) == -4
    assert decode(lib, size=need, weights=FAKE) == -4   # the scores have no room
    assert more >= need + 4 * 16 * 640 * 4
    assert decode(lib, size=more - 1, weights=FAKE) == -4


def test_workspace_size(lib):
    d = gdn.make_attn_dims(**A)
    assert gdn.gdn_attn_decode_kv8_workspace_size(d, 0) % 256 == 0
    for bad in (dict(n=-1), dict(n=1, capacity=-64), dict(n=1, capacity=65), dict(n=1 << 30, capacity=1 << 30)):
        assert gdn.gdn_attn_decode_kv8_workspace_size(d, **bad) == 0, bad
    assert gdn.gdn_attn_decode_kv8_workspace_size(gdn.make_attn_dims(**dict(A, d=96)), 1) == 0
    assert gdn.gdn_attn_decode_kv8_workspace_size(gdn.make_attn_dims(**dict(A, page_size=8)), 1) == 0


def evict(lib, dims=None, c=None, w=FAKE, lens=FAKE, n=4, keep=100, first=0, last=0, to=None,
          w_out=FAKE + 4096, new=FAKE + 4096, kept=FAKE):
    d = dims or gdn.make_attn_dims(**A)
    return lib.gdn_kv8_evict(ctypes.byref(d), _binding._ref(c or cache()), w, lens, n, keep, first, last,
                             _binding._ref(to or cache()), w_out, new, kept, None, None)


def test_evict_refusals(lib):
    for kw, rc in BAD16 + BAD_PAGES:
        assert evict(lib, gdn.make_attn_dims(**kw)) == rc, kw
    for kw, rc in BAD_CACHES:
        assert evict(lib, c=cache(**kw)) == rc, kw
        assert evict(lib, to=cache(**kw)) == rc, kw
    assert evict(lib, n=0) == 0
    assert evict(lib, n=-1) == -1
    assert evict(lib, n=9) == -1
    assert evict(lib, to=cache(seqs=3)) == -1
    assert evict(lib, keep=0) == -1
    assert evict(lib, first=-1) == -1
    assert evict(lib, last=-1) == -1
    assert evict(lib, first=60, last=41) == -1
    assert evict(lib, first=(1 << 31) - 1, last=(1 << 31) - 1) == -1
    assert evict(lib, keep=641) == -1                   # the new pages hold 640
    assert evict(lib, w=None) == -1
    assert evict(lib, lens=None) == -1
    assert evict(lib, new=None) == -1
    assert evict(lib, kept=None) == -1
    assert evict(lib, w_out=FAKE) == -1                 # in place
    assert evict(lib, new=FAKE) == -1
    assert evict(lib, w=FAKE + 4) == -5


def test_sections():
    assert gdn.rope_sections([2, 1, 1]) == [0, 0, 1, 2]
    assert gdn.rope_sections([4, 2, 1], interleaved=True) == [0, 1, 2, 0, 1, 0, 0]
    assert gdn.rope_sections([0, 2]) == [1, 1]
    with pytest.raises(ValueError):
        gdn.rope_sections([1, -1])
    a = gdn.make_rope_axes([0, 2, 1, 0])
    assert a.count == 3 and list(a.pair[:5]) == [0, 2, 1, 0, 0]
    assert gdn.make_rope_axes([]).count == 1
    for bad in ([4], [-1], [0] * 129):
        with pytest.raises(ValueError):
            gdn.make_rope_axes(bad)


def _tensors(pages=3, h=2, page=16, d=64, **kw):
    t = dict(k=torch.zeros(pages, h, page, d, dtype=torch.uint8).view(torch.float8_e4m3fn),
             v=torch.zeros(pages, h, page, d, dtype=torch.uint8).view(torch.float8_e4m3fn),
             k_scale=torch.zeros(pages, h, page // 16), v_scale=torch.zeros(pages, h, page // 16),
             block_table=torch.zeros(1, 2, dtype=torch.int32))
    t.update(kw)
    return t


def test_a_caches_tensors_are_checked(lib):
    gdn.Kv8Cache(**_tensors())
    for kw, what in ((dict(k=torch.zeros(3, 2, 16, 64)), TypeError),
                     (dict(v=torch.zeros(3, 2, 16, 32, dtype=torch.float8_e4m3fn)), ValueError),
                     (dict(k_scale=torch.zeros(3, 2, 2)), ValueError),
                     (dict(v_scale=torch.zeros(3, 2, 1, dtype=torch.float64)), TypeError),
                     (dict(block_table=torch.zeros(1, 2)), TypeError),
                     (dict(block_table=torch.zeros(2, dtype=torch.int32)), ValueError),
                     (dict(page=24, k_scale=torch.zeros(3, 2, 1)), ValueError)):
        with pytest.raises(what):
            gdn.Kv8Cache(**_tensors(**kw))
    k = torch.zeros(3, 2, 64, 16, dtype=torch.uint8).view(torch.float8_e4m3fn).transpose(2, 3)
    with pytest.raises(ValueError, match="contiguous"):
        gdn.Kv8Cache(**_tensors(k=k))
    c = gdn.Kv8Cache(**_tensors())
    other = c._replace(block_table=torch.zeros(5, 7, dtype=torch.int32))
    assert other.block_table.shape == (5, 7) and other.handle != c.handle and other.k is c.k


def test_host_tensors_and_other_shapes_are_refused(lib):
    c = gdn.Kv8Cache(**_tensors())
    dims = gdn.make_attn_dims(4, 2, 64, page_size=16)
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_kv8_gather(dims, c, ints, 0)
    with pytest.raises(ValueError, match=r"cache.k must be \[num_pages, 4, 16, 64\]"):
        gdn.gdn_kv8_gather(gdn.make_attn_dims(4, 4, 64, page_size=16), c, ints, 0)
    with pytest.raises(TypeError, match="Kv8Cache"):
        gdn.gdn_kv8_gather(dims, tuple(c), ints, 0)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="weights has"):
        gdn.gdn_attn_decode_kv8(dims, q, c, ints[:1], None, weights=torch.zeros(1, 2, 16))
    with pytest.raises(ValueError, match="weights_out has"):
        gdn.gdn_kv8_evict(dims, c, torch.zeros(1, 2, 32), ints[:1], 16, c, torch.zeros(1, 2, 16))
    with pytest.raises(ValueError, match="keep does not fit"):
        gdn.gdn_kv8_evict(dims, c, torch.zeros(1, 2, 32), ints[:1], 1 << 31, c)
    with pytest.raises(TypeError, match="gdn_rope_axes"):
        gdn.gdn_qk_norm_rope_axes(dims, q, None, None, None, None, ints, None)
    with pytest.raises(ValueError, match="positions has"):
        gdn.gdn_kv8_append(dims, q, q[:, :2], q[:, :2], None, None, None, ints, c, ints[:1],
                           axes=gdn.make_rope_axes([0, 1, 2]))
    with pytest.raises(ValueError, match="cu_seqlens has"):
        gdn.gdn_kv8_append(dims, q, q[:, :2], q[:, :2], None, None, None, ints[:1], c, ints[:1],
                           cu_seqlens=ints[:1])


def test_a_copied_or_moved_cache(lib):
    """A copy's calls go to the copy's tensors; a tensor given other memory is refused."""
    import copy
    c = gdn.Kv8Cache(**_tensors())
    d = copy.deepcopy(c)
    assert isinstance(d, gdn.Kv8Cache) and d.k.data_ptr() != c.k.data_ptr() and d.handle != c.handle
    assert copy.copy(c).handle == c.handle
    dims, ints = gdn.make_attn_dims(4, 2, 64, page_size=16), torch.zeros(2, dtype=torch.int32)
    d.handle = c.handle
    with pytest.raises(ValueError, match="another than when it was made"):
        gdn.gdn_kv8_gather(dims, d, ints, 0)
    c.k_scale.data = torch.zeros(3, 2, 1)
    with pytest.raises(ValueError, match="another than when it was made"):
        gdn.gdn_kv8_gather(dims, c, ints, 0)
