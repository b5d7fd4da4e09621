"""The marshalling of the 8-bit cache's calls on a host without a GPU, with the stand-ins of
test_attn_marshalling: on which device and stream a call goes, where its outputs are
allocated, what it refuses, and the arguments that reach the library."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from gated_deltanet_linear_07_gb300 import _binding
from tests.test_attn_marshalling import CURRENT, D, HKV, HQ, N, PAGE, SIDE, Tensor, _ints
from tests.test_attn_marshalling import calls as attn_calls  # noqa: F401

NAMES = ("axes", "append", "gather", "decode", "evict")
F8 = torch.float8_e4m3fn


@pytest.fixture
def calls(attn_calls):  # noqa: F811
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    signatures = ([P] * 6 + [I64, P, P, P], [P] * 9 + [I32, I64] + [P] * 5,
                  [P] * 3 + [I32, I64] + [P] * 4, [P] * 4 + [I32] + [P] * 4 + [ctypes.c_size_t, P, P],
                  [P] * 4 + [I32] * 4 + [P] * 6)
    keep = []
    for name, args in zip(NAMES, signatures):
        def entry(*a, name=name):
            attn_calls.seen.append((name, a[-1] or 0))
            attn_calls.args = a
            if name == "axes":
                attn_calls.axes = gdn.gdn_rope_axes.from_buffer_copy(ctypes.string_at(a[2], 132))
            if name == "append":
                size = ctypes.sizeof(gdn.gdn_kv8_cache)
                attn_calls.cache = gdn.gdn_kv8_cache.from_buffer_copy(ctypes.string_at(a[11], size))
            return 0
        keep.append(ctypes.CFUNCTYPE(ctypes.c_int, *args)(entry))
    _binding._calls.setup_kv8(F8, tuple(ctypes.cast(f, P).value for f in keep))
    attn_calls.keep8 = keep
    yield attn_calls


def _cache(device=0, seqs=N, odd=None):
    def on(name):
        return 1 if name == odd else device
    return gdn.Kv8Cache(Tensor((5, HKV, PAGE, D), F8, on("k")), Tensor((5, HKV, PAGE, D), F8, on("v")),
                        Tensor((5, HKV, 1), torch.float32, on("k_scale")),
                        Tensor((5, HKV, 1), torch.float32, on("v_scale")),
                        _ints(seqs, 2, device=on("block_table")))


def _call(name, device=0, odd=None, **kw):
    def on(arg):
        return 1 if arg == odd else device
    dims = gdn.make_attn_dims(HQ, HKV, D, page_size=PAGE)
    q, k, v = (Tensor((N, h, D), device=on(a)) for a, h in (("q", HQ), ("k", HKV), ("v", HKV)))
    c = _cache(on("cache"))
    if "status" in kw:
        kw["d_status"] = _ints(1, device=on(kw.pop("status")))
    lens = _ints(N, device=on("lens"))
    weights = Tensor((N, HKV, 2 * PAGE), torch.float32, on("weights"))
    if name == "axes":
        return gdn.gdn_qk_norm_rope_axes(dims, q, k, None, None, None, _ints(3, N, device=on("positions")),
                                         gdn.make_rope_axes([0, 1, 2]), **kw)
    if name == "append":
        return gdn.gdn_kv8_append(dims, q, k, v, None, None, None, lens, c, lens, **kw)
    if name == "gather":
        return gdn.gdn_kv8_gather(dims, c, lens, 7, **kw)
    if name == "decode":
        return gdn.gdn_attn_decode_kv8(dims, q, c, lens, Tensor((1 << 20,), torch.uint8, on("workspace")),
                                       weights=weights, **kw)
    return gdn.gdn_kv8_evict(dims, c, weights, lens, 20, _cache(on("to")), **kw)


@pytest.mark.parametrize("name", NAMES)
def test_the_current_stream_and_its_memory_by_default(calls, name):
    _call(name)
    assert calls.seen[-1] == (name, CURRENT)
    assert set(calls.seen[:-1]) == {("empty", "current")}


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("stream", [SIDE, 0])
def test_outputs_of_a_call_on_another_stream_come_from_its_memory(calls, name, stream):
    _call(name, stream=stream)
    assert calls.seen[-1] == (name, stream)
    assert set(calls.seen[:-1]) == {("empty", stream)}


@pytest.mark.parametrize("name,odd", [("axes", "k"), ("axes", "positions"), ("append", "v"),
                                      ("append", "cache"), ("append", "lens"), ("gather", "cache"),
                                      ("decode", "cache"), ("decode", "workspace"),
                                      ("decode", "weights"), ("evict", "to"), ("evict", "weights")])
def test_tensors_of_two_devices_are_refused(calls, name, odd):
    with pytest.raises(ValueError, match="cuda:[01]"):
        _call(name, odd=odd)
    assert not any(e[0] == name for e in calls.seen)


@pytest.mark.parametrize("odd", ["k", "v", "k_scale", "v_scale", "block_table"])
def test_a_cache_of_two_devices_is_refused(calls, odd):
    with pytest.raises(ValueError, match="one device"):
        _cache(odd=odd)


@pytest.mark.parametrize("name", NAMES)
def test_another_device_than_the_current_one_is_refused(calls, name):
    with pytest.raises(ValueError, match="current device is cuda:0"):
        _call(name, device=1)
    assert calls.seen == []
    calls.device = 1
    _call(name, device=1)
    assert calls.seen[-1] == (name, CURRENT + 1)


@pytest.mark.parametrize("name", NAMES)
def test_a_status_word_elsewhere_is_refused(calls, name):
    with pytest.raises(ValueError, match="d_status is on cuda:1|cuda:0"):
        _call(name, odd="status", status="status")
    assert not any(e[0] == name for e in calls.seen)


def test_what_reaches_the_library(calls):
    q, k = _call("axes")
    assert calls.args[6] == N and q.shape == (N, HQ, D) and k.shape == (N, HKV, D)
    assert calls.axes.count == 3 and list(calls.axes.pair[:4]) == [0, 1, 2, 0]
    q = _call("append")
    assert calls.args[9] == N and calls.args[10] == N and calls.args[7] is None and calls.args[2] is None
    c = calls.cache
    assert (c.num_pages, c.num_seqs, c.pages_per_seq) == (5, N, 2)
    k, v = _call("gather")
    assert calls.args[3] == N - 1 and calls.args[4] == 7 and k.shape == v.shape == (7, HKV, D)
    o = _call("decode")
    assert calls.args[4] == N and calls.args[9] == 1 << 20 and o.shape == (N, HQ, D)
    lens, kept = _call("evict", first=3, last=5)
    assert calls.args[4:8] == (N, 20, 3, 5) and lens.shape == (N,) and kept.shape == (N, HKV, 20)
    assert calls.args[9] is None and kept.dtype == torch.int32
