"""The attention calls' marshalling on a host without a GPU: stand-ins for
device tensors, for torch's functions and for the library's entry points.  On
which device and stream a call goes, where its outputs are allocated, and what
it refuses."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from gated_deltanet_linear_07_gb300 import _binding

N, HQ, HKV, D, PAGE = 3, 4, 2, 64, 16
CURRENT, SIDE = 0x1000, 0x2000


class Tensor:
    """What the module asks of a tensor."""

    def __init__(self, shape, dtype=torch.bfloat16, device=0):
        like = torch.empty(shape, device="meta", dtype=dtype)
        self.shape, self.dtype, self.device = like.shape, dtype, f"cuda:{device}"
        self._stride, self._numel, self._index = like.stride(), like.numel(), device
        self.is_cuda = True

    def stride(self):
        return self._stride

    def numel(self):
        return self._numel

    def data_ptr(self):
        return 1 << 20

    def is_contiguous(self):
        return True

    def get_device(self):
        return self._index

    def element_size(self):
        return self.dtype.itemsize


@pytest.fixture
def calls(monkeypatch):
    """The module with fakes under it; .seen: (entry point, stream) and ("empty", stream)."""
    gdn.build()
    real = _binding._attn_calls()
    monkeypatch.setattr(_binding, "_calls", real)
    seen = []

    class State:
        device = 0
    state = State()
    state.seen = seen
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    signatures = ([P] * 5 + [I64, P, P, P], [P] * 7 + [I64] + [P] * 5,
                  [P] * 6 + [I32, I64, I64] + [P] * 4,
                  [P] * 4 + [I32, I64] + [P] * 3 + [ctypes.c_size_t, P, P])
    keep = []
    for name, args in zip(("norm_rope", "append", "prefill", "decode"), signatures):
        def entry(*a, name=name):
            seen.append((name, a[-1] or 0))
            return 0
        keep.append(ctypes.CFUNCTYPE(ctypes.c_int, *args)(entry))

    def empty(size, dtype, device):
        seen.append(("empty", "current"))
        return Tensor(size, dtype, state.device)

    def empty_on(size, dtype, device, stream):
        seen.append(("empty", int(stream)))
        return Tensor(size, dtype, state.device)
    real.setup((torch.float32, torch.bfloat16, torch.float16), torch.int32, torch.float64, empty,
               empty_on, lambda device: CURRENT + device, lambda: state.device, gdn.GdnError,
               tuple(ctypes.cast(f, P).value for f in keep))
    state.keep = keep
    yield state
    monkeypatch.setattr(_binding, "_calls", None)    # the next call sets it up anew
    _binding._attn_calls()


def _ints(*shape, device=0):
    return Tensor(shape, torch.int32, device)


def _call(name, device=0, odd=None, **kw):
    """One call on stand-ins; odd: the argument that is on device 1."""
    def on(arg):
        return 1 if arg == odd else device
    dims = gdn.make_attn_dims(HQ, HKV, D, page_size=PAGE)
    q, k, v = (Tensor((N, h, D), device=on(a)) for a, h in (("q", HQ), ("k", HKV), ("v", HKV)))
    kc, vc = (Tensor((5, HKV, PAGE, D), device=on(a)) for a in ("k_cache", "v_cache"))
    pos, table = _ints(N, device=on("positions")), _ints(N, 2, device=on("block_table"))
    if "status" in kw:
        kw["d_status"] = _ints(1, device=on(kw.pop("status")))
    if "o" in kw:
        kw["o"] = Tensor((N, HQ, D), device=on("o"))
    if name == "norm_rope":
        return gdn.gdn_qk_norm_rope(dims, q, k, None, None, None, pos, **kw)
    if name == "append":
        return gdn.gdn_kv_append(dims, q, k, v, None, None, None, pos, kc, vc, table, **kw)
    if name == "prefill":
        return gdn.gdn_attn_prefill(dims, q, k, v, pos, **kw)
    return gdn.gdn_attn_decode(dims, q, kc, vc, table, pos,
                               Tensor((1 << 20,), torch.uint8, on("workspace")), **kw)


NAMES = ("norm_rope", "append", "prefill", "decode")


@pytest.mark.parametrize("name", NAMES)
def test_the_current_stream_and_its_memory_by_default(calls, name):
    _call(name)
    assert calls.seen[-1] == (name, CURRENT)
    assert set(calls.seen[:-1]) == {("empty", "current")}
    calls.seen.clear()
    _call(name, stream=CURRENT)
    assert calls.seen[-1] == (name, CURRENT)
    assert set(calls.seen[:-1]) == {("empty", "current")}


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("stream", [SIDE, 0])
def test_outputs_of_a_call_on_another_stream_come_from_its_memory(calls, name, stream):
    _call(name, stream=stream)
    assert calls.seen[-1] == (name, stream)
    assert set(calls.seen[:-1]) == {("empty", stream)}


def test_a_given_output_is_taken_on_any_stream(calls):
    _call("prefill", o=True, stream=SIDE)
    assert calls.seen == [("prefill", SIDE)]


@pytest.mark.parametrize("name,odd", [("norm_rope", "k"), ("norm_rope", "positions"), ("append", "v"),
                                      ("append", "k_cache"), ("append", "block_table"),
                                      ("prefill", "q"), ("prefill", "v"), ("decode", "v_cache"),
                                      ("decode", "workspace")])
def test_tensors_of_two_devices_are_refused(calls, name, odd):
    with pytest.raises(ValueError, match="cuda:1"):
        _call(name, odd=odd)
    assert not any(e[0] == name for e in calls.seen)


@pytest.mark.parametrize("name", NAMES)
def test_an_output_or_status_word_elsewhere_is_refused(calls, name):
    with pytest.raises(ValueError, match="d_status is on cuda:1"):
        _call(name, odd="status", status="status")
    if name in ("prefill", "decode"):
        with pytest.raises(ValueError, match="o is on cuda:1"):
            _call(name, odd="o", o=True)
    assert not any(e[0] == name for e in calls.seen)


@pytest.mark.parametrize("name", NAMES)
def test_another_device_than_the_current_one_is_refused(calls, name):
    with pytest.raises(ValueError, match="current device is cuda:0"):
        _call(name, device=1)
    assert calls.seen == []
    calls.device = 1
    _call(name, device=1)
    assert calls.seen[-1] == (name, CURRENT + 1)
