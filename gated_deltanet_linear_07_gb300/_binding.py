"""Thin ctypes binding of libgdn_gb300.so (include/gdn.h), same names as the C
ABI.  It only marshals arguments: shapes and device pointers of torch tensors
go in, a non-zero gdn_status comes back as GdnError.  Every step of the layer
runs in the library's CUDA kernels; there is no Python or CPU fallback, and
loading fails loudly when the library has not been built."""
from __future__ import annotations

import ctypes
import os
from typing import Any, NamedTuple

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgdn_gb300.so")

GDN_FP32, GDN_BF16, GDN_FP16 = 0, 1, 2
GDN_DEV_BAD_SLOT, GDN_DEV_BAD_CU_SEQLENS, GDN_DEV_WAIT_TIMEOUT = 0x1, 0x2, 0x4
GDN_FP32_STATE = 0x1   # gdn_dims.flags: fp32 state products in prefill
GDN_CHECK_FINITE = 0x2  # gdn_dims.flags: per-stage NaN/Inf probe of prefill
GDN_TEST_WAIT_TIMEOUT = 0x4  # gdn_dims.flags (tests only): 2 ms waits, one chunk withheld
GDN_BF16_OPERANDS = 0x8      # gdn_dims.flags: bf16 instead of fp16 tensor-core operands
GDN_DEV_NONFINITE_FRONTEND, GDN_DEV_NONFINITE_CHUNK, GDN_DEV_NONFINITE_OUT = 0x8, 0x10, 0x20
GDN_DEV_BAD_PAGE, GDN_DEV_BAD_LENGTH = 0x40, 0x80   # full attention over a paged cache
GDN_ROPE_HALF, GDN_ROPE_INTERLEAVED = 0, 1
STATUS = {0: "GDN_OK", -1: "GDN_EINVAL", -2: "GDN_EUNSUPPORTED", -3: "GDN_ECUDA",
          -4: "GDN_EWORKSPACE", -5: "GDN_EALIGN"}

_lib = None


class GdnError(RuntimeError):
    def __init__(self, func: str, status: int):
        self.status = status
        msg = _lib.gdn_status_str(status).decode() if _lib is not None else ""
        super().__init__(f"{func} returned {STATUS.get(status, status)} ({msg})")


class gdn_dims(ctypes.Structure):
    _fields_ = [("h_k", ctypes.c_int32), ("h_v", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("conv_w", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("io", ctypes.c_int32), ("l2_eps", ctypes.c_float), ("flags", ctypes.c_int32)]


class gdn_params(ctypes.Structure):
    _fields_ = [("conv_weight", ctypes.c_void_p), ("A_log", ctypes.c_void_p),
                ("dt_bias", ctypes.c_void_p)]


class gdn_attn_dims(ctypes.Structure):
    _fields_ = [("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("io", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("rope", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("norm_eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("flags", ctypes.c_int32)]


class gdn_view(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class gdn_rope_params(ctypes.Structure):
    _fields_ = [("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p), ("rope_scale", ctypes.c_float),
                ("d_status", ctypes.c_void_p)]


class gdn_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("num_seqs", ctypes.c_int32),
                ("pages_per_seq", ctypes.c_int32)]


GDN_ROPE_MAX_AXES, GDN_KV8_BLOCK = 4, 16


class gdn_rope_axes(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int32), ("pair", ctypes.c_uint8 * 128)]


class gdn_kv8_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("num_seqs", ctypes.c_int32),
                ("pages_per_seq", ctypes.c_int32)]


GDN_NUM_STAGES = 3
STAGES = ("frontend", "chunk", "scan")


class gdn_trace(ctypes.Structure):
    _fields_ = [("begin", ctypes.c_void_p * GDN_NUM_STAGES),
                ("end", ctypes.c_void_p * GDN_NUM_STAGES),
                ("launches", ctypes.c_int32), ("stages_run", ctypes.c_int32)]


def make_dims(h_k, h_v, d_k, d_v, chunk=64, io="bf16", conv_w=4, l2_eps=1e-6,
              flags=0) -> gdn_dims:
    io_code = {"fp32": GDN_FP32, "bf16": GDN_BF16}[io] if isinstance(io, str) else int(io)
    return gdn_dims(h_k, h_v, d_k, d_v, conv_w, chunk, io_code, l2_eps, flags)


def dims_from(d) -> gdn_dims:
    """gdn_dims from any object with h_k, h_v, d_k, d_v, chunk, io, conv_w, l2_eps
    (and optionally flags)."""
    if isinstance(d, gdn_dims):
        return d
    return make_dims(d.h_k, d.h_v, d.d_k, d.d_v, d.chunk, d.io, d.conv_w, d.l2_eps,
                     getattr(d, "flags", 0))


def load() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    D, PR = ctypes.POINTER(gdn_dims), ctypes.POINTER(gdn_params)
    lib.gdn_status_str.argtypes = [ctypes.c_int]
    lib.gdn_status_str.restype = ctypes.c_char_p
    lib.gdn_conv1d_update.argtypes = [D, P, P, P, I64, P, I32, P, P, P]
    lib.gdn_conv1d_update.restype = ctypes.c_int
    lib.gdn_prefill_workspace_size.argtypes = [D, I64, I32]
    lib.gdn_prefill_workspace_size.restype = SZ
    lib.gdn_prefill.argtypes = [D, PR, P, P, P, P, I32, I64, P, P, P, P, I64, P, P, SZ, P, P]
    lib.gdn_prefill.restype = ctypes.c_int
    lib.gdn_prefill_traced.argtypes = [D, PR, P, P, P, P, I32, I64, P, P, P, P, I64, P, P, SZ, P,
                                       ctypes.POINTER(gdn_trace), P]
    lib.gdn_prefill_traced.restype = ctypes.c_int
    lib.gdn_prefill_noalloc.argtypes = [D, PR, P, P, P, P, I32, I64, P, P, P, P, I64, P, P, P]
    lib.gdn_prefill_noalloc.restype = ctypes.c_int
    lib.gdn_decode_step.argtypes = [D, PR, P, P, P, P, I32, P, P, I64, P, P, P]
    lib.gdn_decode_step.restype = ctypes.c_int
    lib.gdn_gated_rmsnorm.argtypes = [D, P, ctypes.c_float, P, P, I64, P, P]
    lib.gdn_gated_rmsnorm.restype = ctypes.c_int
    lib.gdn_prefill_checkpointed.argtypes = [D, PR, P, P, P, P, I32, I64, P, P, P, P, I64, P, P,
                                             SZ, I64, P, P, P]
    lib.gdn_prefill_checkpointed.restype = ctypes.c_int
    lib.gdn_slot_copy.argtypes = [D, P, P, I64, P, P, I32, P, P]
    lib.gdn_slot_copy.restype = ctypes.c_int
    F = ctypes.c_float
    lib.gdn_prefill_gated_norm.argtypes = [D, PR, P, P, P, P, I32, I64, P, P, P, P, I64, P, P, F,
                                           P, P, SZ, P, P]
    lib.gdn_prefill_gated_norm.restype = ctypes.c_int
    lib.gdn_decode_step_gated_norm.argtypes = [D, PR, P, P, P, P, I32, P, P, I64, P, P, F, P, P, P]
    lib.gdn_decode_step_gated_norm.restype = ctypes.c_int
    lib.gdn_gate_projection.argtypes = [D, P, P, I32, I64, P, P, P, P]
    lib.gdn_gate_projection.restype = ctypes.c_int
    A, V = ctypes.POINTER(gdn_attn_dims), ctypes.POINTER(gdn_view)
    RP, KV = ctypes.POINTER(gdn_rope_params), ctypes.POINTER(gdn_kv_cache)
    lib.gdn_qk_norm_rope.argtypes = [A, RP, V, V, P, I64, P, P, P]
    lib.gdn_qk_norm_rope.restype = ctypes.c_int
    lib.gdn_kv_append.argtypes = [A, RP, V, V, V, P, P, I64, KV, P, P, P, P]
    lib.gdn_kv_append.restype = ctypes.c_int
    lib.gdn_attn_prefill.argtypes = [A, V, V, V, P, P, I32, I64, I64, V, P, P, P]
    lib.gdn_attn_prefill.restype = ctypes.c_int
    lib.gdn_attn_decode_workspace_size.argtypes = [A, I32, I64]
    lib.gdn_attn_decode_workspace_size.restype = SZ
    lib.gdn_attn_decode.argtypes = [A, V, KV, P, I32, I64, V, P, P, SZ, P, P]
    lib.gdn_attn_decode.restype = ctypes.c_int
    X, K8 = ctypes.POINTER(gdn_rope_axes), ctypes.POINTER(gdn_kv8_cache)
    lib.gdn_qk_norm_rope_axes.argtypes = [A, RP, X, V, V, P, I64, P, P, P]
    lib.gdn_qk_norm_rope_axes.restype = ctypes.c_int
    lib.gdn_kv8_append.argtypes = [A, RP, X, V, V, V, P, P, P, I32, I64, K8, P, P, P, P]
    lib.gdn_kv8_append.restype = ctypes.c_int
    lib.gdn_kv8_gather.argtypes = [A, K8, P, I32, I64, P, P, P, P]
    lib.gdn_kv8_gather.restype = ctypes.c_int
    lib.gdn_attn_decode_kv8_workspace_size.argtypes = [A, I32, I64]
    lib.gdn_attn_decode_kv8_workspace_size.restype = SZ
    lib.gdn_attn_decode_kv8.argtypes = [A, V, K8, P, I32, V, P, P, P, SZ, P, P]
    lib.gdn_attn_decode_kv8.restype = ctypes.c_int
    lib.gdn_kv8_evict.argtypes = [A, K8, P, P, I32, I32, I32, I32, K8, P, P, P, P, P]
    lib.gdn_kv8_evict.restype = ctypes.c_int
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(int(stream))
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(func, rc):
    if rc != 0:
        raise GdnError(func, rc)


def _io_dtype(d: gdn_dims):
    import torch
    return torch.bfloat16 if d.io == GDN_BF16 else torch.float32


def _expect(t, name, dtype=None, numel=None):
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")


def conv_dim(d: gdn_dims) -> int:
    return 2 * d.h_k * d.d_k + d.h_v * d.d_v


def gdn_prefill_workspace_size(dims, total_tokens: int, num_seqs: int) -> int:
    d = dims_from(dims)
    return int(load().gdn_prefill_workspace_size(ctypes.byref(d), int(total_tokens), int(num_seqs)))


def gdn_conv1d_update(dims, conv_weight, x, conv_pool, slot_idx, y, d_status=None, stream=None):
    import torch
    d = dims_from(dims)
    n = int(slot_idx.numel())
    io = _io_dtype(d)
    _expect(conv_weight, "conv_weight", torch.float32, conv_dim(d) * d.conv_w)
    _expect(x, "x", io, n * conv_dim(d))
    _expect(y, "y", io, n * conv_dim(d))
    _expect(conv_pool, "conv_pool", io)
    _expect(slot_idx, "slot_idx", torch.int32)
    num_slots = conv_pool.numel() // ((d.conv_w - 1) * conv_dim(d))
    rc = load().gdn_conv1d_update(ctypes.byref(d), _ptr(conv_weight), _ptr(x), _ptr(conv_pool),
                                  num_slots, _ptr(slot_idx), n, _ptr(y), _ptr(d_status),
                                  _stream(stream))
    _check("gdn_conv1d_update", rc)


def gdn_prefill(dims, conv_weight, A_log, dt_bias, x, a, b, cu_seqlens, slot_idx,
                has_initial_state, state_pool, conv_pool, o, workspace, d_status=None,
                stream=None, trace=None):
    """Whole layer over a varlen batch (see gdn_prefill in include/gdn.h).

    trace: optional gdn_trace (stage events + launch count); when given the call
    goes through gdn_prefill_traced."""
    import torch
    d = dims_from(dims)
    io = _io_dtype(d)
    B = int(cu_seqlens.numel()) - 1
    T = int(x.shape[0]) if x is not None else 0
    cd = conv_dim(d)
    _expect(conv_weight, "conv_weight", torch.float32, cd * d.conv_w)
    _expect(A_log, "A_log", torch.float32, d.h_v)
    _expect(dt_bias, "dt_bias", torch.float32, d.h_v)
    _expect(x, "x", io, T * cd)
    _expect(a, "a", io, T * d.h_v)
    _expect(b, "b", io, T * d.h_v)
    _expect(o, "o", io, T * d.h_v * d.d_v)
    _expect(cu_seqlens, "cu_seqlens", torch.int32)
    _expect(slot_idx, "slot_idx", torch.int32, B)
    _expect(has_initial_state, "has_initial_state", torch.uint8, B)
    _expect(state_pool, "state_pool", torch.float32)
    _expect(conv_pool, "conv_pool", io)
    num_slots = state_pool.numel() // (d.h_v * d.d_k * d.d_v)
    p = gdn_params(conv_weight.data_ptr(), A_log.data_ptr(), dt_bias.data_ptr())
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (ctypes.byref(d), ctypes.byref(p), _ptr(x), _ptr(a), _ptr(b), _ptr(cu_seqlens), B, T,
            _ptr(slot_idx), _ptr(has_initial_state), _ptr(state_pool), _ptr(conv_pool),
            num_slots, _ptr(o), _ptr(workspace), ws_bytes, _ptr(d_status))
    if trace is None:
        _check("gdn_prefill", load().gdn_prefill(*args, _stream(stream)))
    else:
        _check("gdn_prefill_traced",
               load().gdn_prefill_traced(*args, ctypes.byref(trace), _stream(stream)))


def gdn_prefill_checkpointed(dims, conv_weight, A_log, dt_bias, x, a, b, cu_seqlens, slot_idx,
                             has_initial_state, state_pool, conv_pool, o, workspace, ckpt_every,
                             ckpt_slot, d_status=None, stream=None):
    """gdn_prefill plus interval checkpoints: every ckpt_every tokens (a multiple
    of the chunk) strictly inside sequence b, its state and conv window go to
    slot ckpt_slot[b] + k - 1 (see gdn_prefill_checkpointed in include/gdn.h)."""
    import torch
    d = dims_from(dims)
    io = _io_dtype(d)
    B = int(cu_seqlens.numel()) - 1
    T = int(x.shape[0]) if x is not None else 0
    cd = conv_dim(d)
    _expect(conv_weight, "conv_weight", torch.float32, cd * d.conv_w)
    _expect(A_log, "A_log", torch.float32, d.h_v)
    _expect(dt_bias, "dt_bias", torch.float32, d.h_v)
    _expect(x, "x", io, T * cd)
    _expect(a, "a", io, T * d.h_v)
    _expect(b, "b", io, T * d.h_v)
    _expect(o, "o", io, T * d.h_v * d.d_v)
    _expect(cu_seqlens, "cu_seqlens", torch.int32)
    _expect(slot_idx, "slot_idx", torch.int32, B)
    _expect(has_initial_state, "has_initial_state", torch.uint8, B)
    _expect(ckpt_slot, "ckpt_slot", torch.int32, B)
    _expect(state_pool, "state_pool", torch.float32)
    _expect(conv_pool, "conv_pool", io)
    num_slots = state_pool.numel() // (d.h_v * d.d_k * d.d_v)
    p = gdn_params(conv_weight.data_ptr(), A_log.data_ptr(), dt_bias.data_ptr())
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("gdn_prefill_checkpointed", load().gdn_prefill_checkpointed(
        ctypes.byref(d), ctypes.byref(p), _ptr(x), _ptr(a), _ptr(b), _ptr(cu_seqlens), B, T,
        _ptr(slot_idx), _ptr(has_initial_state), _ptr(state_pool), _ptr(conv_pool), num_slots,
        _ptr(o), _ptr(workspace), ws_bytes, int(ckpt_every), _ptr(ckpt_slot), _ptr(d_status),
        _stream(stream)))


def gdn_prefill_gated_norm(dims, conv_weight, A_log, dt_bias, x, a, b, cu_seqlens, slot_idx,
                           has_initial_state, state_pool, conv_pool, z, norm_weight, y, workspace,
                           eps=1e-6, d_status=None, stream=None):
    """gdn_prefill with the gated RMSNorm of the output fused in: writes
    y = rmsnorm(o) * norm_weight * SiLU(z) (see gdn_prefill_gated_norm in
    include/gdn.h)."""
    import torch
    d = dims_from(dims)
    io = _io_dtype(d)
    B = int(cu_seqlens.numel()) - 1
    T = int(x.shape[0]) if x is not None else 0
    cd = conv_dim(d)
    _expect(conv_weight, "conv_weight", torch.float32, cd * d.conv_w)
    _expect(A_log, "A_log", torch.float32, d.h_v)
    _expect(dt_bias, "dt_bias", torch.float32, d.h_v)
    _expect(x, "x", io, T * cd)
    _expect(a, "a", io, T * d.h_v)
    _expect(b, "b", io, T * d.h_v)
    _expect(z, "z", io, T * d.h_v * d.d_v)
    _expect(y, "y", io, T * d.h_v * d.d_v)
    _expect(norm_weight, "norm_weight", torch.float32, d.d_v)
    _expect(cu_seqlens, "cu_seqlens", torch.int32)
    _expect(slot_idx, "slot_idx", torch.int32, B)
    _expect(has_initial_state, "has_initial_state", torch.uint8, B)
    _expect(state_pool, "state_pool", torch.float32)
    _expect(conv_pool, "conv_pool", io)
    num_slots = state_pool.numel() // (d.h_v * d.d_k * d.d_v)
    p = gdn_params(conv_weight.data_ptr(), A_log.data_ptr(), dt_bias.data_ptr())
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("gdn_prefill_gated_norm", load().gdn_prefill_gated_norm(
        ctypes.byref(d), ctypes.byref(p), _ptr(x), _ptr(a), _ptr(b), _ptr(cu_seqlens), B, T,
        _ptr(slot_idx), _ptr(has_initial_state), _ptr(state_pool), _ptr(conv_pool), num_slots,
        _ptr(z), _ptr(norm_weight), float(eps), _ptr(y), _ptr(workspace), ws_bytes,
        _ptr(d_status), _stream(stream)))


def gdn_decode_step_gated_norm(dims, conv_weight, A_log, dt_bias, x, a, b, slot_idx, state_pool,
                               conv_pool, z, norm_weight, y, eps=1e-6, d_status=None, stream=None):
    """gdn_decode_step with the gated RMSNorm of the output fused in (see
    gdn_decode_step_gated_norm in include/gdn.h)."""
    import torch
    d = dims_from(dims)
    io = _io_dtype(d)
    n = int(slot_idx.numel())
    cd = conv_dim(d)
    _expect(conv_weight, "conv_weight", torch.float32, cd * d.conv_w)
    _expect(A_log, "A_log", torch.float32, d.h_v)
    _expect(dt_bias, "dt_bias", torch.float32, d.h_v)
    _expect(x, "x", io, n * cd)
    _expect(a, "a", io, n * d.h_v)
    _expect(b, "b", io, n * d.h_v)
    _expect(z, "z", io, n * d.h_v * d.d_v)
    _expect(y, "y", io, n * d.h_v * d.d_v)
    _expect(norm_weight, "norm_weight", torch.float32, d.d_v)
    _expect(slot_idx, "slot_idx", torch.int32, n)
    _expect(state_pool, "state_pool", torch.float32)
    _expect(conv_pool, "conv_pool", io)
    num_slots = state_pool.numel() // (d.h_v * d.d_k * d.d_v)
    p = gdn_params(conv_weight.data_ptr(), A_log.data_ptr(), dt_bias.data_ptr())
    _check("gdn_decode_step_gated_norm", load().gdn_decode_step_gated_norm(
        ctypes.byref(d), ctypes.byref(p), _ptr(x), _ptr(a), _ptr(b), _ptr(slot_idx), n,
        _ptr(state_pool), _ptr(conv_pool), num_slots, _ptr(z), _ptr(norm_weight), float(eps),
        _ptr(y), _ptr(d_status), _stream(stream)))


def gdn_slot_copy(dims, state_pool, conv_pool, src_slot, dst_slot, d_status=None, stream=None):
    """Copy whole slots (state and conv window): slot dst_slot[i] <- slot
    src_slot[i]; padding pairs (< 0) skipped (see gdn_slot_copy in include/gdn.h)."""
    import torch
    d = dims_from(dims)
    _expect(state_pool, "state_pool", torch.float32)
    _expect(conv_pool, "conv_pool", _io_dtype(d))
    n = int(src_slot.numel())
    _expect(src_slot, "src_slot", torch.int32, n)
    _expect(dst_slot, "dst_slot", torch.int32, n)
    num_slots = state_pool.numel() // (d.h_v * d.d_k * d.d_v)
    _check("gdn_slot_copy", load().gdn_slot_copy(
        ctypes.byref(d), _ptr(state_pool), _ptr(conv_pool), num_slots, _ptr(src_slot),
        _ptr(dst_slot), n, _ptr(d_status), _stream(stream)))


GDN_NOALLOC_SCRATCH_BYTES = 64 << 20


def gdn_prefill_noalloc(dims, conv_weight, A_log, dt_bias, x, a, b, cu_seqlens, slot_idx,
                        has_initial_state, state_pool, conv_pool, o, d_status=None, stream=None):
    """gdn_prefill without a workspace argument, for callers that cannot allocate
    device memory: the library uses its own fixed device scratch array of
    GDN_NOALLOC_SCRATCH_BYTES (see gdn_prefill_noalloc in include/gdn.h)."""
    import torch
    d = dims_from(dims)
    io = _io_dtype(d)
    B = int(cu_seqlens.numel()) - 1
    T = int(x.shape[0]) if x is not None else 0
    cd = conv_dim(d)
    _expect(conv_weight, "conv_weight", torch.float32, cd * d.conv_w)
    _expect(A_log, "A_log", torch.float32, d.h_v)
    _expect(dt_bias, "dt_bias", torch.float32, d.h_v)
    _expect(x, "x", io, T * cd)
    _expect(a, "a", io, T * d.h_v)
    _expect(b, "b", io, T * d.h_v)
    _expect(o, "o", io, T * d.h_v * d.d_v)
    _expect(cu_seqlens, "cu_seqlens", torch.int32)
    _expect(slot_idx, "slot_idx", torch.int32, B)
    _expect(has_initial_state, "has_initial_state", torch.uint8, B)
    _expect(state_pool, "state_pool", torch.float32)
    _expect(conv_pool, "conv_pool", io)
    num_slots = state_pool.numel() // (d.h_v * d.d_k * d.d_v)
    p = gdn_params(conv_weight.data_ptr(), A_log.data_ptr(), dt_bias.data_ptr())
    rc = load().gdn_prefill_noalloc(ctypes.byref(d), ctypes.byref(p), _ptr(x), _ptr(a), _ptr(b),
                                    _ptr(cu_seqlens), B, T, _ptr(slot_idx),
                                    _ptr(has_initial_state), _ptr(state_pool), _ptr(conv_pool),
                                    num_slots, _ptr(o), _ptr(d_status), _stream(stream))
    _check("gdn_prefill_noalloc", rc)


def make_trace(begin_events=None, end_events=None) -> gdn_trace:
    """gdn_trace from lists (per stage) of torch.cuda.Event or None."""
    tr = gdn_trace()
    for i in range(GDN_NUM_STAGES):
        for dst, evs in ((tr.begin, begin_events), (tr.end, end_events)):
            ev = evs[i] if evs is not None else None
            dst[i] = ev.cuda_event if ev is not None else None
    return tr


def gdn_decode_step(dims, conv_weight, A_log, dt_bias, x, a, b, slot_idx, state_pool,
                    conv_pool, o, d_status=None, stream=None):
    """One decode token per row (see gdn_decode_step in include/gdn.h)."""
    import torch
    d = dims_from(dims)
    io = _io_dtype(d)
    n = int(slot_idx.numel())
    cd = conv_dim(d)
    _expect(conv_weight, "conv_weight", torch.float32, cd * d.conv_w)
    _expect(A_log, "A_log", torch.float32, d.h_v)
    _expect(dt_bias, "dt_bias", torch.float32, d.h_v)
    _expect(x, "x", io, n * cd)
    _expect(a, "a", io, n * d.h_v)
    _expect(b, "b", io, n * d.h_v)
    _expect(o, "o", io, n * d.h_v * d.d_v)
    _expect(slot_idx, "slot_idx", torch.int32)
    _expect(state_pool, "state_pool", torch.float32)
    _expect(conv_pool, "conv_pool", io)
    num_slots = state_pool.numel() // (d.h_v * d.d_k * d.d_v)
    p = gdn_params(conv_weight.data_ptr(), A_log.data_ptr(), dt_bias.data_ptr())
    rc = load().gdn_decode_step(ctypes.byref(d), ctypes.byref(p), _ptr(x), _ptr(a), _ptr(b),
                                _ptr(slot_idx), n, _ptr(state_pool), _ptr(conv_pool), num_slots,
                                _ptr(o), _ptr(d_status), _stream(stream))
    _check("gdn_decode_step", rc)


def gdn_gated_rmsnorm(dims, weight, o, z, y=None, eps=1e-6, stream=None):
    """Gated RMSNorm of the layer output (see gdn_gated_rmsnorm in
    include/gdn.h): o, z [n, h_v, d_v] in the I/O dtype, weight [d_v] fp32;
    y defaults to o (in place).  Returns y."""
    import torch
    d = dims_from(dims)
    io = _io_dtype(d)
    n = int(o.numel()) // (d.h_v * d.d_v) if d.h_v * d.d_v else 0
    y = o if y is None else y
    _expect(weight, "weight", torch.float32, d.d_v)
    _expect(o, "o", io, n * d.h_v * d.d_v)
    _expect(z, "z", io, n * d.h_v * d.d_v)
    _expect(y, "y", io, n * d.h_v * d.d_v)
    rc = load().gdn_gated_rmsnorm(ctypes.byref(d), _ptr(weight), float(eps), _ptr(o), _ptr(z), n,
                                  _ptr(y), _stream(stream))
    _check("gdn_gated_rmsnorm", rc)
    return y


def gdn_gate_projection(dims, hidden, w_ba, a=None, b=None, d_status=None, stream=None):
    """The decay and beta input projections as one matmul (see
    gdn_gate_projection in include/gdn.h): hidden [n, d_model] bf16, w_ba
    [2 h_v, d_model] bf16 (decay rows, then beta rows) -> a, b [n, h_v] bf16
    (allocated when not given).  Returns (a, b)."""
    import torch
    d = dims_from(dims)
    if hidden.dim() != 2:
        raise ValueError("hidden must be [n, d_model]")
    n, d_model = int(hidden.shape[0]), int(hidden.shape[1])
    if a is None:
        a = torch.empty((n, d.h_v), dtype=torch.bfloat16, device=hidden.device)
    if b is None:
        b = torch.empty((n, d.h_v), dtype=torch.bfloat16, device=hidden.device)
    _expect(hidden, "hidden", torch.bfloat16)
    _expect(w_ba, "w_ba", torch.bfloat16, 2 * d.h_v * d_model)
    _expect(a, "a", torch.bfloat16, n * d.h_v)
    _expect(b, "b", torch.bfloat16, n * d.h_v)
    _expect(d_status, "d_status", torch.int32, 1)
    rc = load().gdn_gate_projection(ctypes.byref(d), _ptr(hidden), _ptr(w_ba), d_model, n,
                                    _ptr(a), _ptr(b), _ptr(d_status), _stream(stream))
    _check("gdn_gate_projection", rc)
    return a, b


# ---- full attention ---------------------------------------------------------


def make_attn_dims(h_q, h_kv, d, io="bf16", rot_dim=0, rope="half", page_size=64, norm_eps=1e-6,
                   scale=None, flags=0) -> gdn_attn_dims:
    """gdn_attn_dims: scale None is 1 / sqrt(d)."""
    io_code = {"fp32": GDN_FP32, "bf16": GDN_BF16, "fp16": GDN_FP16}[io] if isinstance(io, str) \
        else int(io)
    rope_code = {"half": GDN_ROPE_HALF, "interleaved": GDN_ROPE_INTERLEAVED}[rope] \
        if isinstance(rope, str) else int(rope)
    return gdn_attn_dims(h_q, h_kv, d, io_code, rot_dim, rope_code, page_size, norm_eps,
                         0.0 if scale is None else scale, flags)


def rope_frequencies(rot_dim, theta=1e4, scaling=None, factor=1.0, original_len=None,
                     beta_fast=32.0, beta_slow=1.0, device="cpu"):
    """(inv_freq, rope_scale) for gdn_qk_norm_rope and gdn_kv_append: the
    frequencies theta^(-2 i / rot_dim) in fp64 (radians per position), scaled
    for contexts `factor` times as long as the trained `original_len`:
      None      as trained;
      "linear"  every frequency divided by factor (positions interpolated);
      "ntk"     theta raised to theta * factor^(rot_dim / (rot_dim - 2)), so
                that the highest frequency stays and the lowest is interpolated;
      "yarn"    frequencies that turn more than beta_fast times over
                original_len stay, those that turn less than beta_slow times
                are interpolated, a linear ramp between (Peng et al., YaRN);
                rope_scale = 0.1 ln(factor) + 1."""
    import math

    import torch
    if rot_dim % 2 or rot_dim < 2:
        raise ValueError(f"rot_dim must be even and positive, got {rot_dim}")
    if not theta > 0 or not factor > 0:
        raise ValueError("theta and factor must be positive")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs rot_dim >= 4")
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    freq = theta ** (-2.0 * i / rot_dim)
    rope_scale = 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if original_len is None or not original_len > 0 or not beta_fast > beta_slow > 0:
            raise ValueError("yarn scaling needs original_len > 0 and beta_fast > beta_slow > 0")

        def index(turns):   # the (fractional) pair that turns this often over original_len
            return rot_dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo = max(math.floor(index(beta_fast)), 0)
        hi = min(math.ceil(index(beta_slow)), rot_dim - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        freq = freq / factor * (1 - keep) + freq * keep
        rope_scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.to(device), rope_scale


_calls = None


def _attn_calls():
    """The marshalling module of the attention calls, handed the library's entry
    points (its shape, type and layout checks raise as this module's do)."""
    global _calls
    if _calls is None:
        import importlib.util

        import torch

        from ._build import CALLS
        lib = load()
        if not os.path.exists(CALLS):
            raise ImportError(f"{CALLS} is missing: build it first "
                              "(python -c 'import __graft_entry__ as g; g.build()')")
        spec = importlib.util.spec_from_file_location(f"{__package__}._attn_calls", CALLS)
        calls = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(calls)
        fns = (lib.gdn_qk_norm_rope, lib.gdn_kv_append, lib.gdn_attn_prefill, lib.gdn_attn_decode)
        # the raw handle of a device's current stream; current_stream() builds an object first
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
        device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        calls.setup((torch.float32, torch.bfloat16, torch.float16), torch.int32, torch.float64,
                    torch.empty, _empty_on, raw, device, GdnError,
                    tuple(ctypes.cast(f, ctypes.c_void_p).value for f in fns))
        fns = (lib.gdn_qk_norm_rope_axes, lib.gdn_kv8_append, lib.gdn_kv8_gather,
               lib.gdn_attn_decode_kv8, lib.gdn_kv8_evict)
        calls.setup_kv8(torch.float8_e4m3fn,
                        tuple(ctypes.cast(f, ctypes.c_void_p).value for f in fns))
        _calls = calls
    return _calls


def _empty_on(size, dtype, device, stream):
    """torch.empty from the memory of the stream with this handle."""
    import torch
    handle = int(stream)
    s = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(s):
        return torch.empty(size, dtype=dtype, device=device)


def _ref(v):
    return None if v is None else ctypes.byref(v)


def gdn_qk_norm_rope(dims, q, k, q_norm, k_norm, inv_freq, positions, q_out=None, k_out=None,
                     rope_scale=1.0, stream=None, d_status=None):
    """Per-head norm and rotation of queries and keys (see gdn_qk_norm_rope in
    include/gdn.h): q [n, h_q, d], k [n, h_kv, d] (either may be None), norm
    weights [d] fp32 or None, inv_freq [rot_dim / 2] fp64, positions [n] int32.
    Outputs are allocated when not given.  Returns (q_out, k_out)."""
    return (_calls or _attn_calls()).qk_norm_rope(dims, q, k, q_norm, k_norm, inv_freq, positions,
                                                  q_out, k_out, rope_scale, d_status, stream)


def gdn_kv_append(dims, q, k, v, q_norm, k_norm, inv_freq, positions, k_cache, v_cache, block_table,
                  row_seq=None, q_out=None, k_out=None, rope_scale=1.0, d_status=None, stream=None):
    """gdn_qk_norm_rope with the keys, and the values, going into the paged
    cache (see gdn_kv_append in include/gdn.h): caches [num_pages, h_kv,
    page_size, d], block_table [num_seqs, pages_per_seq] int32, row_seq [n]
    int32 (None: row t is sequence t), k_out [n, h_kv, d] or None (packed keys
    too, for a prompt's attention).  Returns q_out (None when q is None)."""
    return (_calls or _attn_calls()).kv_append(dims, q, k, v, q_norm, k_norm, inv_freq, positions,
                                               k_cache, v_cache, block_table, row_seq, q_out, k_out,
                                               rope_scale, d_status, stream)


def gdn_attn_prefill(dims, q, k, v, cu_seqlens, cu_seqlens_kv=None, gate=None, o=None,
                     d_status=None, stream=None):
    """Causal attention over packed prompts (see gdn_attn_prefill in
    include/gdn.h): q [total_q, h_q, d], k, v [total_kv, h_kv, d], cu_seqlens
    [num_seqs + 1] int32 (cu_seqlens_kv None: the same for the keys), gate
    [total_q, h_q, d] or None.  o is allocated when not given.  Returns o."""
    return (_calls or _attn_calls()).attn_prefill(dims, q, k, v, cu_seqlens, cu_seqlens_kv, gate, o,
                                                  d_status, stream)


def gdn_attn_decode_workspace_size(dims, n: int, shared_len: int = 0) -> int:
    return int(load().gdn_attn_decode_workspace_size(ctypes.byref(dims), int(n), int(shared_len)))


def gdn_attn_decode(dims, q, k_cache, v_cache, block_table, seq_lens, workspace, shared_len=0,
                    gate=None, o=None, d_status=None, stream=None):
    """One query token per sequence against the paged cache (see
    gdn_attn_decode in include/gdn.h): q [n, h_q, d], caches [num_pages, h_kv,
    page_size, d], block_table [num_seqs, pages_per_seq] int32, seq_lens [n]
    int32; the first shared_len tokens (whole pages) are common to all rows.
    o is allocated when not given.  Returns o."""
    return (_calls or _attn_calls()).attn_decode(dims, q, k_cache, v_cache, block_table, seq_lens,
                                                 workspace, int(shared_len), gate, o, d_status,
                                                 stream)


# ---- positions with several axes, the cache held in 8 bits --------------------


def rope_sections(sections, interleaved=False):
    """The axis of each pair of channels, for make_rope_axes: sections[a] pairs for
    axis a, one section after the other, or, interleaved, taking turns as long
    as a section lasts (0, 1, 2, 0, 1, 2, ..., 0, 0)."""
    left = [int(s) for s in sections]
    if any(s < 0 for s in left):
        raise ValueError("sections must not be negative")
    if not interleaved:
        return [a for a, s in enumerate(left) for _ in range(s)]
    out = []
    while any(left):
        for a, s in enumerate(left):
            if s:
                out.append(a)
                left[a] -= 1
    return out


def make_rope_axes(axis_of_pair, count=None) -> gdn_rope_axes:
    """gdn_rope_axes from the axis of each pair of channels (rot_dim / 2 of them; see
    rope_sections).  count: the axes that positions have, where that is more than
    the pairs use (None: up to the last one that a pair turns by)."""
    axis = [int(a) for a in axis_of_pair]
    if len(axis) > 128 or any(not 0 <= a < GDN_ROPE_MAX_AXES for a in axis):
        raise ValueError(f"at most 128 pairs, of axes 0 to {GDN_ROPE_MAX_AXES - 1}")
    used = max(axis, default=0) + 1
    count = used if count is None else int(count)
    if not used <= count <= GDN_ROPE_MAX_AXES:
        raise ValueError(f"count must be {used} (the pairs') to {GDN_ROPE_MAX_AXES}, got {count}")
    return gdn_rope_axes(count, (ctypes.c_uint8 * 128)(*axis))


class _Kv8Tensors(NamedTuple):
    k: Any             # [num_pages, h_kv, page_size, d] float8_e4m3fn
    v: Any
    k_scale: Any       # [num_pages, h_kv, page_size / 16] fp32
    v_scale: Any
    block_table: Any   # [num_seqs, pages_per_seq] int32


class Kv8Cache(_Kv8Tensors):
    """A paged cache held in 8 bits (see gdn_kv8_cache in include/gdn.h): (k, v, k_scale,
    v_scale, block_table).  Made once for its tensors, whose shapes and addresses it keeps
    for the calls (they may be written to, not moved: ValueError)."""

    def __new__(cls, k, v, k_scale, v_scale, block_table):
        self = super().__new__(cls, k, v, k_scale, v_scale, block_table)
        self.handle = (_calls or _attn_calls()).kv8_make(k, v, k_scale, v_scale, block_table)
        return self

    @classmethod
    def _make(cls, tensors):
        return cls(*tensors)

    def __reduce__(self):   # a copy's tensors have addresses of their own
        return Kv8Cache, tuple(self)


def make_kv8_cache(dims, num_pages, block_table) -> Kv8Cache:
    """A Kv8Cache of zeros beside block_table ([num_seqs, pages_per_seq] int32)."""
    import torch
    dev = block_table.device
    shape = (int(num_pages), dims.h_kv, dims.page_size, dims.d)

    def codes():
        return torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)

    def scales():
        return torch.zeros((*shape[:2], dims.page_size // GDN_KV8_BLOCK), device=dev)
    return Kv8Cache(codes(), codes(), scales(), scales(), block_table)


def gdn_qk_norm_rope_axes(dims, q, k, q_norm, k_norm, inv_freq, positions, axes, q_out=None,
                          k_out=None, rope_scale=1.0, stream=None, d_status=None):
    """gdn_qk_norm_rope with a position on each of several axes (see
    gdn_qk_norm_rope_axes in include/gdn.h): positions [axes' count, n] int32,
    axes from make_rope_axes.  Returns (q_out, k_out)."""
    return (_calls or _attn_calls()).qk_norm_rope_axes(dims, q, k, q_norm, k_norm, inv_freq,
                                                       positions, axes, q_out, k_out, rope_scale,
                                                       d_status, stream)


def gdn_kv8_append(dims, q, k, v, q_norm, k_norm, inv_freq, positions, cache, starts,
                   cu_seqlens=None, axes=None, q_out=None, k_out=None, rope_scale=1.0,
                   d_status=None, stream=None):
    """Norm and rotate q and k, and store k and v in an 8-bit cache (see
    gdn_kv8_append in include/gdn.h): positions [n] or [axes' count, n] int32, cache a
    Kv8Cache, starts [num_seqs] int32 (tokens that each sequence holds already),
    cu_seqlens [num_seqs + 1] int32 (None: row t is sequence t), k_out [n, h_kv, d]
    or None.  Returns q_out (None when q is None)."""
    return (_calls or _attn_calls()).kv8_append(dims, q, k, v, q_norm, k_norm, inv_freq, positions,
                                                cache, starts, cu_seqlens, axes, q_out, k_out,
                                                rope_scale, d_status, stream)


def gdn_kv8_gather(dims, cache, cu_seqlens, total, k_out=None, v_out=None, d_status=None,
                   stream=None):
    """The cached tokens as packed keys and values (see gdn_kv8_gather in
    include/gdn.h): row cu_seqlens[b] + p is place p of sequence b, total =
    cu_seqlens[-1] rows.  Returns (k, v), each [total, h_kv, d]."""
    return (_calls or _attn_calls()).kv8_gather(dims, cache, cu_seqlens, int(total), k_out, v_out,
                                                d_status, stream)


def gdn_attn_decode_kv8_workspace_size(dims, n: int, capacity: int = 0) -> int:
    """capacity: tokens of a block table row where weights are collected, else 0."""
    return int(load().gdn_attn_decode_kv8_workspace_size(ctypes.byref(dims), int(n), int(capacity)))


def gdn_attn_decode_kv8(dims, q, cache, seq_lens, workspace, gate=None, weights=None, o=None,
                        d_status=None, stream=None):
    """One query token per sequence against an 8-bit cache (see
    gdn_attn_decode_kv8 in include/gdn.h): q [n, h_q, d], seq_lens [n] int32; weights
    [num_seqs, h_kv, pages_per_seq * page_size] fp32, to which what each cached token
    receives is added, or None.  Returns o."""
    return (_calls or _attn_calls()).attn_decode_kv8(dims, q, cache, seq_lens, workspace, gate,
                                                     weights, o, d_status, stream)


def gdn_kv8_evict(dims, cache, weights, seq_lens, keep, to, weights_out=None, first=0, last=0,
                  new_lens=None, kept=None, d_status=None, stream=None):
    """Cut sequences down to `keep` cached tokens each, copied to the pages of the
    Kv8Cache `to`: the first and last ones and those with the greatest weights (see
    gdn_kv8_evict in include/gdn.h).  Returns (new_lens [n], kept [n, h_kv, keep])."""
    return (_calls or _attn_calls()).kv8_evict(dims, cache, weights, seq_lens, int(keep), to,
                                               weights_out, int(first), int(last), new_lens, kept,
                                               d_status, stream)
