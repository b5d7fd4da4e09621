"""Full attention: what the entry points refuse, on a host without a GPU (every
call below fails validation or has nothing to do, and never reaches the CUDA
runtime), the binding's checks of its tensors, and the rotation frequencies."""
import ctypes
import math

import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from gated_deltanet_linear_07_gb300 import _binding

FAKE = 1 << 20   # an aligned, never-dereferenced address
A = dict(h_q=16, h_kv=4, d=256, rot_dim=64)


@pytest.fixture(scope="module")
def lib():
    gdn.build()
    return gdn.load()


def view(data=FAKE, ts=4096, hs=256):
    return gdn.gdn_view(data, ts, hs)


BAD_DIMS = [(dict(A, h_q=15), -1), (dict(A, h_kv=0), -1), (dict(A, d=96), -2), (dict(A, io=7), -2),
            (dict(A, rot_dim=24), -2), (dict(A, rot_dim=272), -2), (dict(A, rot_dim=-16), -2),
            (dict(A, norm_eps=float("nan")), -1), (dict(A, norm_eps=-1.0), -1),
            (dict(A, scale=-1.0), -1), (dict(A, scale=float("nan")), -1), (dict(A, rope=2), -1),
            (dict(A, flags=1), -1)]


def norm_rope(lib, dims=None, q=view(), k=view(hs=256), pos=FAKE, n=4, q_out=FAKE, k_out=FAKE,
              freq=FAKE, qn=FAKE, scale=1.0):
    p = gdn.gdn_rope_params(qn, FAKE, freq, scale)
    d = dims or gdn.make_attn_dims(**A)
    return lib.gdn_qk_norm_rope(ctypes.byref(d), ctypes.byref(p), _binding._ref(q), _binding._ref(k),
                                pos, n, q_out, k_out, None)


def test_norm_rope_refusals(lib):
    for kw, rc in BAD_DIMS:
        assert norm_rope(lib, gdn.make_attn_dims(**kw)) == rc, kw
    assert norm_rope(lib, n=-1) == -1
    assert norm_rope(lib, n=0) == 0
    assert norm_rope(lib, n=1 << 31) == -2
    assert norm_rope(lib, q=None, k=None) == -1
    assert norm_rope(lib, pos=None) == -1
    assert norm_rope(lib, freq=None) == -1
    assert norm_rope(lib, q_out=None) == -1
    assert norm_rope(lib, k_out=None) == -1
    assert norm_rope(lib, scale=float("inf")) == -1
    assert norm_rope(lib, q=view(FAKE + 2)) == -5
    assert norm_rope(lib, q=view(ts=4100)) == -5      # rows not 16-byte aligned
    assert norm_rope(lib, k=view(hs=260)) == -5
    assert norm_rope(lib, k=view(hs=-256)) == -1
    assert norm_rope(lib, k=view(hs=0)) == -2          # a broadcast head
    assert norm_rope(lib, q=view(ts=0)) == -2
    assert norm_rope(lib, qn=FAKE + 4) == -5
    assert norm_rope(lib, k_out=FAKE + 8) == -5
    assert lib.gdn_qk_norm_rope(ctypes.byref(gdn.make_attn_dims(**A)), None, None, None, FAKE, 4,
                                FAKE, FAKE, None) == -1


def cache(k=FAKE, v=FAKE, table=FAKE, pages=100, seqs=8, per=10):
    return gdn.gdn_kv_cache(k, v, table, pages, seqs, per)


BAD_CACHES = [(dict(k=None), -1), (dict(v=None), -1), (dict(table=None), -1), (dict(pages=0), -1),
              (dict(seqs=-1), -1), (dict(per=0), -1), (dict(k=FAKE + 8), -5),
              (dict(pages=1 << 31), -2), (dict(per=1 << 30), -2)]


def append(lib, dims=None, k=view(), v=view(), c=None, n=4, row_seq=FAKE, q_out=FAKE, q=view(),
           k_out=None):
    p = gdn.gdn_rope_params(FAKE, FAKE, FAKE, 1.0)
    d = dims or gdn.make_attn_dims(**A)
    return lib.gdn_kv_append(ctypes.byref(d), ctypes.byref(p), _binding._ref(q), _binding._ref(k),
                             _binding._ref(v), FAKE, row_seq, n, _binding._ref(c or cache()), q_out,
                             k_out, None, None)


def test_append_refusals(lib):
    for kw, rc in BAD_DIMS + [(dict(A, page_size=48), -2), (dict(A, page_size=256), -2)]:
        assert append(lib, gdn.make_attn_dims(**kw)) == rc, kw
    for kw, rc in BAD_CACHES:
        assert append(lib, c=cache(**kw)) == rc, kw
    assert append(lib, n=9, row_seq=None) == -1       # more rows than sequences
    assert append(lib, n=0) == 0
    assert append(lib, k=None) == -1
    assert append(lib, v=None) == -1
    assert append(lib, q_out=None) == -1
    assert append(lib, v=view(FAKE + 4)) == -5
    assert append(lib, k_out=FAKE + 8) == -5


def prefill(lib, dims=None, q=view(), k=view(), v=view(), cu=FAKE, cu_kv=None, B=2, tq=64, tk=64,
            gate=None, o=FAKE + 4096):
    d = dims or gdn.make_attn_dims(**A)
    return lib.gdn_attn_prefill(ctypes.byref(d), _binding._ref(q), _binding._ref(k),
                                _binding._ref(v), cu, cu_kv, B, tq, tk, _binding._ref(gate), o, None,
                                None)


def test_prefill_refusals(lib):
    for kw, rc in BAD_DIMS + [(dict(A, io="fp32"), -2)]:
        assert prefill(lib, gdn.make_attn_dims(**kw)) == rc, kw
    assert prefill(lib, tq=0, tk=0) == 0
    assert prefill(lib, B=0, tq=0, tk=0) == 0
    assert prefill(lib, B=0) == -1
    assert prefill(lib, B=-1) == -1
    assert prefill(lib, tq=-1) == -1
    assert prefill(lib, tk=65) == -1                  # one cu_seqlens for two totals
    assert prefill(lib, q=None) == -1
    assert prefill(lib, k=view(None)) == -1
    assert prefill(lib, cu=None) == -1
    assert prefill(lib, o=None) == -1
    assert prefill(lib, o=FAKE) == -1                 # the output is an input
    assert prefill(lib, o=FAKE + 4100) == -5
    assert prefill(lib, k=view(ts=1028)) == -5
    assert prefill(lib, gate=view(FAKE + 2)) == -5
    assert prefill(lib, tq=1 << 31, tk=1 << 31) == -2
    assert prefill(lib, tq=(1 << 31) - 1, tk=(1 << 31) - 1) == -2   # block ends past 2^31
    assert prefill(lib, v=view(ts=0)) == -2


def decode(lib, dims=None, q=view(), c=None, lens=FAKE, n=4, shared=0, gate=None, o=FAKE + 4096,
           ws=FAKE, ws_bytes=1 << 40):
    d = dims or gdn.make_attn_dims(**A)
    return lib.gdn_attn_decode(ctypes.byref(d), _binding._ref(q), _binding._ref(c or cache()), lens,
                               n, shared, _binding._ref(gate), o, ws, ws_bytes, None, None)


def test_decode_refusals(lib):
    for kw, rc in BAD_DIMS + [(dict(A, io="fp32"), -2), (dict(A, page_size=8), -2)]:
        assert decode(lib, gdn.make_attn_dims(**kw)) == rc, kw
    for kw, rc in BAD_CACHES:
        assert decode(lib, c=cache(**kw)) == rc, kw
    assert decode(lib, n=0) == 0
    assert decode(lib, n=-1) == -1
    assert decode(lib, n=9) == -1                     # more rows than the block table has
    assert decode(lib, shared=32) == -1               # not whole pages
    assert decode(lib, shared=704) == -1              # more than a block table row
    assert decode(lib, shared=-64) == -1
    assert decode(lib, q=None) == -1
    assert decode(lib, lens=None) == -1
    assert decode(lib, o=None) == -1
    assert decode(lib, o=FAKE) == -1
    assert decode(lib, ws=None) == -4
    assert decode(lib, ws_bytes=64) == -4
    assert decode(lib, ws=FAKE + 16) == -5
    assert decode(lib, o=FAKE + 8) == -5
    assert decode(lib, gate=view(hs=12)) == -5


def test_workspace_size_rules(lib):
    d = gdn.make_attn_dims(**A)
    size = gdn.gdn_attn_decode_workspace_size
    assert size(d, 64) > 0 and size(d, 64) % 256 == 0
    assert size(d, 64, 4096) > size(d, 64)            # a prefix leaves partials of its own
    assert size(d, 64, 100) == 0 and size(d, -1) == 0 and size(d, 4, -64) == 0
    assert size(gdn.make_attn_dims(**dict(A, page_size=12)), 4) == 0


def test_binding_checks_its_tensors():
    d = gdn.make_attn_dims(4, 2, 64, io="bf16", rot_dim=32, page_size=16)
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    w, f = torch.ones(64), torch.ones(16, dtype=torch.float64)
    pos = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        gdn.gdn_qk_norm_rope(d, q.float(), k, w, w, f, pos)
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope(d, q[:2], k, w, w, f, pos)
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope(d, q.transpose(1, 2).contiguous().transpose(1, 2), k, w, w, f, pos)
    with pytest.raises(TypeError):
        gdn.gdn_qk_norm_rope(d, q, k, w, w, f.float(), pos)
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope(d, q, k, w[:32], w, f, pos)
    kc = torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_kv_append(d, q, k, k, w, w, f, pos, kc.view(5, 2, 32, 32), kc, table)
    with pytest.raises(TypeError):
        gdn.gdn_kv_append(d, q, k, k, w, w, f, pos, kc, kc, table.long())
    with pytest.raises(ValueError):
        gdn.gdn_attn_prefill(d, q, k, k[:2], pos)
    with pytest.raises(ValueError):
        gdn.gdn_attn_decode(d, q, kc, kc, table, pos[:2], torch.zeros(1))


def test_binding_refuses_host_tensors():
    d = gdn.make_attn_dims(4, 2, 64, rot_dim=0, page_size=16)
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    kc, table = torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(3, 2, dtype=torch.int32)
    for call in (lambda: gdn.gdn_qk_norm_rope(d, q, k, None, None, None, i),
                 lambda: gdn.gdn_kv_append(d, q, k, k, None, None, None, i, kc, kc.clone(), table),
                 lambda: gdn.gdn_attn_prefill(d, q, k, k, i[:2]),
                 lambda: gdn.gdn_attn_decode(d, q, kc, kc, table, i, torch.zeros(1 << 20))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        gdn.gdn_attn_prefill(gdn.make_dims(16, 32, 128, 128), q, k, k, i[:2])


def test_rope_frequencies():
    f, s = gdn.rope_frequencies(64, 1e6)
    assert s == 1.0 and f.dtype == torch.float64 and f[0] == 1.0
    assert math.isclose(float(f[31]), 1e6 ** (-62 / 64), rel_tol=1e-12)
    lin, _ = gdn.rope_frequencies(64, 1e6, "linear", factor=4.0)
    assert torch.allclose(lin * 4, f, rtol=1e-14)
    ntk, _ = gdn.rope_frequencies(64, 1e6, "ntk", factor=4.0)
    assert ntk[0] == 1.0 and math.isclose(float(ntk[31]), float(f[31]) / 4, rel_tol=1e-12)
    yarn, s = gdn.rope_frequencies(64, 1e6, "yarn", factor=4.0, original_len=32768)
    assert math.isclose(s, 0.1 * math.log(4) + 1)
    turns = f * 32768 / (2 * math.pi)
    assert torch.equal(yarn[turns > 64], f[turns > 64])
    assert torch.allclose(yarn[turns < 0.5], f[turns < 0.5] / 4, rtol=1e-14)
    assert ((yarn <= f) & (yarn >= f / 4 * (1 - 1e-12))).all()
    for bad in (dict(rot_dim=63), dict(rot_dim=64, scaling="other"), dict(rot_dim=64, factor=0.0),
                dict(rot_dim=64, scaling="yarn"), dict(rot_dim=64, theta=-1.0)):
        with pytest.raises(ValueError):
            gdn.rope_frequencies(**bad)
