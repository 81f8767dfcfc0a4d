"""ctypes binding of libbdssm.so (the C ABI in include/bdssm.h).

Argument marshalling only: every step of the computation runs in the HIP kernels. The
functions take torch CUDA tensors (PyTorch provides device memory and streams), pass
their device pointers to the library, and raise ``BdssmError`` on a non-OK status.
There is no fallback: if the library is not built, loading raises.
"""
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbdssm.so")

OK, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_ALIGN, ERR_ALIAS, ERR_WORKSPACE, ERR_HIP, ERR_SCRATCH = range(9)
STATIC_SCRATCH_BYTES = 64 << 20
F32, BF16 = 0, 1

# every symbol include/bdssm.h declares
EXPORTS = ("bdssm_abi_version", "bdssm_status_str", "bdssm_prefix_scan_workspace",
           "bdssm_prefix_scan", "bdssm_block_step", "bdssm_block_step_ex", "bdssm_commit",
           "bdssm_decode_graph_create",
           "bdssm_decode_graph_launch", "bdssm_decode_graph_destroy",
           "bdssm_conv_workspace", "bdssm_conv", "bdssm_block_step_conv", "bdssm_commit_conv",
           "bdssm_state_ops_bytes", "bdssm_state_ops", "bdssm_block_step_ops",
           "bdssm_set_launch_override", "bdssm_prefix_scan_static",
           "bdssm_full_window_workspace", "bdssm_full_window",
           "bdssm_state_bf16_bytes", "bdssm_state_bf16", "bdssm_block_step_variant",
           "bdssm_commit_refresh",
           "bdssm_gated_norm", "bdssm_residual_norm",
           "bdssm_attn_step_workspace", "bdssm_attn_step", "bdssm_kv_append",
           "bdssm_attn_step_ex_workspace", "bdssm_attn_step_ex",
           "bdssm_rotary_turns", "bdssm_rotary_step", "bdssm_rotary_append",
           "bdssm_pages_workspace", "bdssm_pages_advance", "bdssm_pages_fork", "bdssm_pages_compact",
           "bdssm_pages_copy")
ROTARY_PLAIN, ROTARY_LINEAR, ROTARY_BASE, ROTARY_PARTS = range(4)
NORM_RMS, NORM_LAYER = 0, 1
STATE_F32, STATE_OPS, STATE_BF16 = 0, 1, 2


class BdssmError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(msg)
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("nheads", ctypes.c_int32),
                ("headdim", ctypes.c_int32), ("d_state", ctypes.c_int32),
                ("ngroups", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32)]


class SeqPtrs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("dt", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("C", ctypes.c_void_p)]


class LaunchOverride(ctypes.Structure):
    _fields_ = [("block_kernel", ctypes.c_int32), ("lat_waves", ctypes.c_int32),
                ("bw_heads", ctypes.c_int32), ("bw_splits", ctypes.c_int32)]


class StepParams(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("D", ctypes.c_void_p), ("A_rev", ctypes.c_void_p),
                ("D_rev", ctypes.c_void_p), ("skip_per_channel", ctypes.c_int32)]


class ConvParams(ctypes.Structure):
    _fields_ = [("width", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class NormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("width", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("rows_per_stream", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class Residual(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("o", ctypes.c_void_p), ("post_w", ctypes.c_void_p),
                ("pre_w", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("gain", ctypes.c_void_p),
                ("shift", ctypes.c_void_p), ("mod_stride", ctypes.c_int64), ("res_scale", ctypes.c_float)]


class AttnDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("nheads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("headdim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class KvCachePtrs(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("max_len", ctypes.c_int32)]


class AttnChunk(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("tokens", ctypes.c_int64), ("starts", ctypes.c_void_p), ("block_len", ctypes.c_int32)]


class AttnMask(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("block", ctypes.c_int32), ("window", ctypes.c_int32),
                ("sinks", ctypes.c_int32)]


class AttnScoresPtrs(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("prefix", ctypes.c_void_p),
                ("first", ctypes.c_void_p), ("last", ctypes.c_void_p)]


class RotaryFreqs(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("kind", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("trained", ctypes.c_int32), ("low", ctypes.c_double), ("high", ctypes.c_double)]


class RotaryPtrs(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float),
                ("turns", ctypes.c_void_p), ("positions", ctypes.c_void_p)]


class RotaryOut(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64)]


class PagesDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


class PagesPtrs(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("uses", ctypes.c_void_p)]


_lib = None


def load():
    """Load the built library (raises OSError if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OSError(f"{LIB_PATH} is not built; run bidirectional_mamba_state_amd/build.py")
        lib = ctypes.CDLL(LIB_PATH)
        V, P, I32, I64, SZ = ctypes.c_void_p, ctypes.POINTER, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        lib.bdssm_abi_version.restype = ctypes.c_int
        lib.bdssm_abi_version.argtypes = []
        lib.bdssm_status_str.restype = ctypes.c_char_p
        lib.bdssm_status_str.argtypes = [ctypes.c_int]
        lib.bdssm_prefix_scan_workspace.restype = SZ
        lib.bdssm_prefix_scan_workspace.argtypes = [P(Dims), I64, I32, I32, I32]
        lib.bdssm_prefix_scan.restype = ctypes.c_int
        lib.bdssm_prefix_scan.argtypes = [P(Dims), I64, I32, P(SeqPtrs), V, V, V, V, V, V, V, SZ, V]
        lib.bdssm_block_step.restype = ctypes.c_int
        lib.bdssm_block_step.argtypes = [P(Dims), I32, V, P(SeqPtrs), P(SeqPtrs), V, V, V, V]
        lib.bdssm_block_step_ex.restype = ctypes.c_int
        lib.bdssm_block_step_ex.argtypes = [P(Dims), I32, V, P(SeqPtrs), P(SeqPtrs), V, V, V, V, V, V]
        lib.bdssm_commit.restype = ctypes.c_int
        lib.bdssm_commit.argtypes = [P(Dims), I32, P(SeqPtrs), V, V, V, V, V]
        lib.bdssm_decode_graph_create.restype = ctypes.c_int
        lib.bdssm_state_ops_bytes.restype = SZ
        lib.bdssm_state_ops_bytes.argtypes = [P(Dims)]
        lib.bdssm_state_ops.restype = ctypes.c_int
        lib.bdssm_state_ops.argtypes = [P(Dims), V, V, V]
        lib.bdssm_block_step_ops.restype = ctypes.c_int
        lib.bdssm_block_step_ops.argtypes = [P(Dims), I32, V, P(SeqPtrs), P(SeqPtrs), V, V, V, V, V, V]
        lib.bdssm_decode_graph_create.argtypes = [P(Dims), I32, I32, V, V, P(SeqPtrs), P(SeqPtrs), V, V,
                                                  P(V), P(SeqPtrs), V, V, P(V)]
        lib.bdssm_decode_graph_launch.restype = ctypes.c_int
        lib.bdssm_decode_graph_launch.argtypes = [V, V]
        lib.bdssm_decode_graph_destroy.restype = None
        lib.bdssm_decode_graph_destroy.argtypes = [V]
        lib.bdssm_conv_workspace.restype = SZ
        lib.bdssm_conv_workspace.argtypes = [P(Dims), I64]
        lib.bdssm_conv.restype = ctypes.c_int
        lib.bdssm_conv.argtypes = [P(Dims), I64, P(ConvParams), I32, V, P(SeqPtrs), P(SeqPtrs), V, V]
        lib.bdssm_block_step_conv.restype = ctypes.c_int
        lib.bdssm_block_step_conv.argtypes = [P(Dims), I32, P(ConvParams), P(ConvParams), V, V,
                                              P(SeqPtrs), P(SeqPtrs), V, V, V, V, V, V, SZ, V]
        lib.bdssm_commit_conv.restype = ctypes.c_int
        lib.bdssm_commit_conv.argtypes = [P(Dims), I32, P(ConvParams), P(SeqPtrs), V, V, V, V, V,
                                          V, SZ, V]
        lib.bdssm_prefix_scan_static.restype = ctypes.c_int
        lib.bdssm_prefix_scan_static.argtypes = [P(Dims), I64, I32, P(SeqPtrs), V, V, V, V, V, V, V]
        lib.bdssm_full_window_workspace.restype = SZ
        lib.bdssm_full_window_workspace.argtypes = [P(Dims), I64, I32]
        lib.bdssm_full_window.restype = ctypes.c_int
        lib.bdssm_full_window.argtypes = [P(Dims), I64, I32, P(SeqPtrs), P(SeqPtrs), V, V, V, V, V, V, SZ, V]
        lib.bdssm_state_bf16_bytes.restype = SZ
        lib.bdssm_state_bf16_bytes.argtypes = [P(Dims)]
        lib.bdssm_state_bf16.restype = ctypes.c_int
        lib.bdssm_state_bf16.argtypes = [P(Dims), V, V, V]
        lib.bdssm_block_step_variant.restype = ctypes.c_int
        lib.bdssm_block_step_variant.argtypes = [P(Dims), I32, V, I32, P(SeqPtrs), P(SeqPtrs), P(StepParams), V, V]
        lib.bdssm_commit_refresh.restype = ctypes.c_int
        lib.bdssm_commit_refresh.argtypes = [P(Dims), I32, P(SeqPtrs), V, V, V, V, I32, V, V]
        lib.bdssm_set_launch_override.restype = ctypes.c_int
        lib.bdssm_set_launch_override.argtypes = [P(LaunchOverride)]
        lib.bdssm_gated_norm.restype = ctypes.c_int
        lib.bdssm_gated_norm.argtypes = [P(NormDims), V, V, I64, V, I32, V, V]
        lib.bdssm_residual_norm.restype = ctypes.c_int
        lib.bdssm_residual_norm.argtypes = [P(NormDims), P(Residual), V, V, V]
        lib.bdssm_attn_step_workspace.restype = SZ
        lib.bdssm_attn_step_workspace.argtypes = [P(AttnDims), I32, I32, P(AttnMask)]
        lib.bdssm_attn_step.restype = ctypes.c_int
        lib.bdssm_attn_step.argtypes = [P(AttnDims), P(AttnChunk), P(KvCachePtrs), P(AttnMask), V, V, SZ, V]
        lib.bdssm_kv_append.restype = ctypes.c_int
        lib.bdssm_kv_append.argtypes = [P(AttnDims), P(AttnChunk), P(KvCachePtrs), V, V]
        lib.bdssm_attn_step_ex_workspace.restype = SZ
        lib.bdssm_attn_step_ex_workspace.argtypes = [P(AttnDims), I32, I32, P(AttnMask), P(AttnScoresPtrs)]
        lib.bdssm_attn_step_ex.restype = ctypes.c_int
        lib.bdssm_attn_step_ex.argtypes = [P(AttnDims), P(AttnChunk), P(KvCachePtrs), P(AttnMask), P(AttnScoresPtrs),
                                           V, V, SZ, V]
        lib.bdssm_rotary_turns.restype = ctypes.c_int
        lib.bdssm_rotary_turns.argtypes = [P(RotaryFreqs), V]
        lib.bdssm_rotary_step.restype = ctypes.c_int
        lib.bdssm_rotary_step.argtypes = [P(AttnDims), P(AttnChunk), P(RotaryPtrs), V, P(RotaryOut), V]
        lib.bdssm_rotary_append.restype = ctypes.c_int
        lib.bdssm_rotary_append.argtypes = [P(AttnDims), P(AttnChunk), P(KvCachePtrs), P(RotaryPtrs), P(RotaryOut), V, V]
        lib.bdssm_pages_workspace.restype = SZ
        lib.bdssm_pages_workspace.argtypes = [P(PagesDims)]
        lib.bdssm_pages_advance.restype = ctypes.c_int
        lib.bdssm_pages_advance.argtypes = [P(PagesDims), P(PagesPtrs), V, I32, I32, I32, V, V, V, V, SZ, V]
        lib.bdssm_pages_fork.restype = ctypes.c_int
        lib.bdssm_pages_fork.argtypes = [P(PagesDims), P(PagesPtrs), V, V, V, V, V, V, V, SZ, V]
        lib.bdssm_pages_compact.restype = ctypes.c_int
        lib.bdssm_pages_compact.argtypes = [P(PagesDims), P(PagesPtrs), V, V, V, V, V, SZ, V]
        lib.bdssm_pages_copy.restype = ctypes.c_int
        lib.bdssm_pages_copy.argtypes = [P(AttnDims), P(KvCachePtrs), V, I32, V]
        _lib = lib
    return _lib


def status_str(status):
    return load().bdssm_status_str(status).decode()


def abi_version():
    return load().bdssm_abi_version()


def _check(rc):
    if rc != OK:
        raise BdssmError(rc, status_str(rc))


def _ptr(t):
    """Device pointer of a torch CUDA tensor (None -> NULL). Refuses host tensors and
    non-contiguous views: the library takes contiguous device buffers only."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not getattr(t, "is_cuda", False):
        raise TypeError("bdssm takes device (CUDA/HIP) tensors only")
    if not t.is_contiguous():
        raise ValueError("bdssm takes contiguous tensors only")
    return t.data_ptr()


def _current_stream():
    """A function for the current stream's handle."""
    import torch
    torch.cuda.current_device()  # initializes the device
    raw, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
    if raw is None or device is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    # the same without the Stream object, whose construction takes longer than the rest of a call
    return lambda: raw(device())


_current = None


def _stream(stream):
    global _current
    if stream is None:
        if _current is None:
            _current = _current_stream()
        return _current()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def dims(batch, nheads, headdim, d_state, ngroups, in_dtype, y_dtype=F32):
    return Dims(batch, nheads, headdim, d_state, ngroups, in_dtype, y_dtype)


def _seq(s):
    if s is None:
        return None
    x, dt, B, C = s
    return SeqPtrs(_ptr(x), _ptr(dt), _ptr(B), _ptr(C))


def _byref(v):
    return None if v is None else ctypes.byref(v)


def prefix_scan_workspace(d, length, chunk, with_y, with_chunk_states):
    return load().bdssm_prefix_scan_workspace(ctypes.byref(d), length, chunk, int(with_y),
                                              int(with_chunk_states))


def prefix_scan(d, length, chunk, seq, A, D, h_init, y, chunk_states, h_out,
                workspace=None, workspace_bytes=None, stream=None):
    """bdssm_prefix_scan. seq = (x, dt, B, C) tensors; C may be None when y is None."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().bdssm_prefix_scan(ctypes.byref(d), length, chunk, _byref(_seq(seq)), _ptr(A),
                                    _ptr(D), _ptr(h_init), _ptr(y), _ptr(chunk_states),
                                    _ptr(h_out), _ptr(workspace), workspace_bytes,
                                    _stream(stream)))


def prefix_scan_static(d, length, chunk, seq, A, D, h_init, y, chunk_states, h_out, stream=None):
    """bdssm_prefix_scan_static: bdssm_prefix_scan with its workspace taken from the
    library's static scratch buffer (no workspace argument, nothing allocated)."""
    _check(load().bdssm_prefix_scan_static(ctypes.byref(d), length, chunk, _byref(_seq(seq)), _ptr(A),
                                           _ptr(D), _ptr(h_init), _ptr(y), _ptr(chunk_states),
                                           _ptr(h_out), _stream(stream)))


def full_window_workspace(d, length, chunk):
    return load().bdssm_full_window_workspace(ctypes.byref(d), length, chunk)


def full_window(d, length, chunk, fwd, rev, A, D, A_rev, D_rev, y, workspace=None, stream=None):
    """bdssm_full_window: forward and reverse scans over the whole window from zero states
    (A_rev None = A; D_rev None = no reverse skip term)."""
    _check(load().bdssm_full_window(ctypes.byref(d), length, chunk, _byref(_seq(fwd)), _byref(_seq(rev)),
                                    _ptr(A), _ptr(D), _ptr(A if A_rev is None else A_rev), _ptr(D_rev),
                                    _ptr(y), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def block_step(d, block_len, h_prefix, fwd, rev, A, D, y, stream=None):
    """bdssm_block_step. fwd, rev = (x, dt, B, C) tensors."""
    _check(load().bdssm_block_step(ctypes.byref(d), block_len, _ptr(h_prefix), _byref(_seq(fwd)),
                                   _byref(_seq(rev)), _ptr(A), _ptr(D), _ptr(y), _stream(stream)))


def block_step_ex(d, block_len, h_prefix, fwd, rev, A, D, A_rev, D_rev, y, stream=None):
    """bdssm_block_step_ex: separate reverse-direction decay A_rev and skip weight D_rev
    (None = no reverse skip term)."""
    _check(load().bdssm_block_step_ex(ctypes.byref(d), block_len, _ptr(h_prefix), _byref(_seq(fwd)),
                                      _byref(_seq(rev)), _ptr(A), _ptr(D), _ptr(A_rev), _ptr(D_rev),
                                      _ptr(y), _stream(stream)))


def state_ops_bytes(d):
    """bdssm_state_ops_bytes (SIZE_MAX for invalid or unsupported dims)."""
    return load().bdssm_state_ops_bytes(ctypes.byref(d))


def state_ops(d, h, ops, stream=None):
    """bdssm_state_ops: the cached state h in operand form, into ops."""
    _check(load().bdssm_state_ops(ctypes.byref(d), _ptr(h), _ptr(ops), _stream(stream)))


def block_step_ops(d, block_len, h_ops, fwd, rev, A, D, y, A_rev=None, D_rev=None, stream=None):
    """bdssm_block_step_ops: block step from the state in operand form (A_rev None = A)."""
    _check(load().bdssm_block_step_ops(ctypes.byref(d), block_len, _ptr(h_ops), _byref(_seq(fwd)),
                                       _byref(_seq(rev)), _ptr(A), _ptr(D),
                                       _ptr(A if A_rev is None else A_rev), _ptr(D_rev), _ptr(y),
                                       _stream(stream)))


KERNEL_AUTO, KERNEL_SMALL_BATCH, KERNEL_BANDWIDTH = 0, 1, 2


def set_launch_override(block_kernel=0, lat_waves=0, bw_heads=0, bw_splits=0):
    """bdssm_set_launch_override (tests and launch-shape sweeps only): pins the block-step
    kernel and its launch shape for later calls; all zeros = automatic."""
    o = LaunchOverride(block_kernel, lat_waves, bw_heads, bw_splits)
    _check(load().bdssm_set_launch_override(ctypes.byref(o)))


def state_bf16_bytes(d):
    """bdssm_state_bf16_bytes (SIZE_MAX for invalid or unsupported dims)."""
    return load().bdssm_state_bf16_bytes(ctypes.byref(d))


def state_bf16(d, h, out, stream=None):
    """bdssm_state_bf16: the bf16 copy of the cached state h, into out."""
    _check(load().bdssm_state_bf16(ctypes.byref(d), _ptr(h), _ptr(out), _stream(stream)))


def block_step_variant(d, block_len, state, state_form, fwd, rev, A, D, y, A_rev=None, D_rev=None,
                       skip_per_channel=False, stream=None):
    """bdssm_block_step_variant: the state as float32, operand form or bf16 (state_form), skip
    weights per head or per channel."""
    prm = StepParams(_ptr(A), _ptr(D), _ptr(A_rev), _ptr(D_rev), int(skip_per_channel))
    _check(load().bdssm_block_step_variant(ctypes.byref(d), block_len, _ptr(state), state_form, _byref(_seq(fwd)),
                                           _byref(_seq(rev)), ctypes.byref(prm), _ptr(y), _stream(stream)))


def commit(d, block_len, clean, A, D, h, y=None, stream=None):
    """bdssm_commit. clean = (x, dt, B, C) tensors (C may be None when y is None)."""
    _check(load().bdssm_commit(ctypes.byref(d), block_len, _byref(_seq(clean)), _ptr(A), _ptr(D),
                               _ptr(h), _ptr(y), _stream(stream)))


def commit_refresh(d, block_len, clean, A, D, h, state_copy, state_form=STATE_OPS, y=None, stream=None):
    """bdssm_commit_refresh: the commit, with the block step's copy of the advanced state
    (operand form or bf16) written in the same pass."""
    _check(load().bdssm_commit_refresh(ctypes.byref(d), block_len, _byref(_seq(clean)), _ptr(A), _ptr(D), _ptr(h),
                                       _ptr(state_copy), state_form, _ptr(y), _stream(stream)))


def conv_params(weight, bias, activation, width=None):
    """A bdssm_conv_params for weight [CH, W] and bias [CH] (or None) device tensors."""
    w = int(weight.shape[1]) if width is None else width
    return ConvParams(w, activation, _ptr(weight), _ptr(bias))


def conv_workspace(d, length):
    return load().bdssm_conv_workspace(ctypes.byref(d), length)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def conv(d, length, params, reverse, state_in, raw, out, state_out, stream=None):
    """bdssm_conv. raw, out = (x, dt, B, C) tensors (dt unused, may be None)."""
    _check(load().bdssm_conv(ctypes.byref(d), length, ctypes.byref(params), int(reverse), _ptr(state_in),
                             _byref(_seq(raw)), _byref(_seq(out)), _ptr(state_out), _stream(stream)))


def block_step_conv(d, block_len, conv_fwd, conv_rev, h_prefix, conv_state, fwd, rev, A, D, y,
                    workspace, A_rev=None, D_rev=None, stream=None):
    """bdssm_block_step_conv: fwd, rev are raw (unconvolved) inputs."""
    _check(load().bdssm_block_step_conv(ctypes.byref(d), block_len, ctypes.byref(conv_fwd),
                                        ctypes.byref(conv_rev), _ptr(h_prefix), _ptr(conv_state),
                                        _byref(_seq(fwd)), _byref(_seq(rev)), _ptr(A), _ptr(D),
                                        _ptr(A_rev), _ptr(D_rev), _ptr(y), _ptr(workspace),
                                        _nbytes(workspace), _stream(stream)))


def commit_conv(d, block_len, params, clean, A, D, h, conv_state, workspace, y=None, stream=None):
    """bdssm_commit_conv: advances h and the conv state in place over raw clean inputs."""
    _check(load().bdssm_commit_conv(ctypes.byref(d), block_len, ctypes.byref(params), _byref(_seq(clean)),
                                    _ptr(A), _ptr(D), _ptr(h), _ptr(conv_state), _ptr(y), _ptr(workspace),
                                    _nbytes(workspace), _stream(stream)))


class DecodeGraph:
    """bdssm_decode_graph_*: the steps of one active block and its commit, recorded once
    and replayed with launch(). Keeps references to the tensors whose addresses it holds."""

    def __init__(self, d, block_len, h, fwd_steps, rev_steps, A, D, ys, clean=None, y_commit=None,
                 h_ops=None):
        import torch
        steps = len(ys)
        if len(fwd_steps) != steps or len(rev_steps) != steps:
            raise ValueError("one fwd, rev and y per step")
        self._keep = (h, h_ops, fwd_steps, rev_steps, A, D, ys, clean, y_commit)
        fw = (SeqPtrs * max(steps, 1))(*[_seq(s) for s in fwd_steps])
        rv = (SeqPtrs * max(steps, 1))(*[_seq(s) for s in rev_steps])
        yp = (ctypes.c_void_p * max(steps, 1))(*[_ptr(t) for t in ys])
        # record on a side stream: the legacy default stream cannot be captured
        side = torch.cuda.Stream()
        handle = ctypes.c_void_p()
        rc = load().bdssm_decode_graph_create(ctypes.byref(d), block_len, steps, _ptr(h), _ptr(h_ops), fw, rv,
                                              _ptr(A), _ptr(D), yp, _byref(_seq(clean)),
                                              _ptr(y_commit), side.cuda_stream, ctypes.byref(handle))
        _check(rc)
        self._handle = handle

    def launch(self, stream=None):
        _check(load().bdssm_decode_graph_launch(self._handle, _stream(stream)))

    def close(self):
        if getattr(self, "_handle", None):
            load().bdssm_decode_graph_destroy(self._handle)
            self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------- norms and attention around the Mamba layers
# A decode step makes these calls for microseconds of GPU work, so their checks are plain
# comparisons of what a tensor already holds.
_torch_dtypes = None  # float32, bfloat16


def _torch_dtype(dtype):
    global _torch_dtypes
    if _torch_dtypes is None:
        import torch
        _torch_dtypes = torch.float32, torch.bfloat16
    return _torch_dtypes[dtype == BF16]


def _expect(t, what, dtype, shape):
    """A tensor argument whose sizes the library cannot see: its type and shape (a tuple)."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{what}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _expect_size(t, what, dtype, shape):
    """Its type and number of elements: rows x width however the tensor splits them."""
    if t.dtype != dtype or t.numel() != shape[0] * shape[1]:
        raise ValueError(f"{what}: expected {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")


def _rows(t, what, dtype, shape):
    """(device pointer, elements between rows) of a tensor of two or three dimensions whose rows
    (all but the first) are contiguous; the rows themselves may be slices of longer ones."""
    if not getattr(t, "is_cuda", False):
        raise TypeError("bdssm takes device (CUDA/HIP) tensors only")
    if t.dtype != dtype or t.shape != shape:
        _expect(t, what, dtype, shape)
    steps, width = t.stride(), shape[-1]
    if len(shape) == 3 and steps[2] == 1 and steps[1] == width:
        return t.data_ptr(), steps[0] if shape[0] > 1 else width * shape[1]
    inside = steps[-1] == 1 or width == 1
    if len(shape) == 3:
        inside = inside and (steps[1] == width or shape[1] == 1)
        width *= shape[1]
    if not inside:
        raise ValueError(f"{what}: rows must be contiguous")
    return t.data_ptr(), steps[0] if shape[0] > 1 else width


_int32 = None


def _expect_int(t, what, shape):
    """An int32 tensor argument: its shape (a tuple)."""
    global _int32
    if _int32 is None:
        import torch
        _int32 = torch.int32
    if t.dtype != _int32 or t.shape != shape:
        _expect(t, what, _int32, shape)


def norm_dims(rows, width, dtype, groups=1, eps=1e-5, rows_per_stream=0, kind=NORM_RMS, x_dtype=None):
    """A bdssm_norm_dims; x_dtype None = dtype."""
    return NormDims(rows, width, groups, rows_per_stream, kind, dtype if x_dtype is None else x_dtype, dtype, eps)


def gated_norm(nd, y, z, weight, out, norm_first=False, stream=None):
    """bdssm_gated_norm: y, out [rows, width] contiguous, z rows of width channels (a slice of
    longer rows is fine), weight [width] float32 or None."""
    dt = _torch_dtype(nd.dtype)
    shape = (nd.rows, nd.width)
    zp, zs = _rows(z, "z", dt, shape)
    _expect_size(y, "y", _torch_dtype(nd.x_dtype), shape)
    _expect_size(out, "out", dt, shape)
    if weight is not None:
        _expect(weight, "weight", _torch_dtype(F32), shape[1:])
    _check(load().bdssm_gated_norm(ctypes.byref(nd), _ptr(y), zp, zs, _ptr(weight), int(norm_first), _ptr(out),
                                   _stream(stream)))


def residual_norm(nd, x, o, pre_w, x_out, u, post_w=None, gate=None, gain=None, shift=None, res_scale=1.0,
                  stream=None):
    """bdssm_residual_norm: x, o, x_out, u [rows, width] contiguous (o, x_out or u may be None),
    post_w, pre_w [width] float32 or None, gate, gain, shift [streams, width] or None (slices of
    one projection's rows)."""
    dt, xt = _torch_dtype(nd.dtype), _torch_dtype(nd.x_dtype)
    shape = (nd.rows, nd.width)
    _expect_size(x, "x", xt, shape)
    if o is not None:
        _expect_size(o, "o", dt, shape)
    if x_out is not None:
        _expect_size(x_out, "x_out", xt, shape)
    if u is not None:
        _expect_size(u, "u", dt, shape)
    if post_w is not None:
        _expect(post_w, "post_w", _torch_dtype(F32), shape[1:])
    if pre_w is not None:
        _expect(pre_w, "pre_w", _torch_dtype(F32), shape[1:])
    gp = ap = sp = None
    step = 0  # between streams
    if gate is not None or gain is not None or shift is not None:
        per = (-(-nd.rows // nd.rows_per_stream) if nd.rows_per_stream > 0 else 0, nd.width)
        steps = []
        if gate is not None:
            gp, step = _rows(gate, "gate", dt, per)
            steps.append(step)
        if gain is not None:
            ap, step = _rows(gain, "gain", dt, per)
            steps.append(step)
        if shift is not None:
            sp, step = _rows(shift, "shift", dt, per)
            steps.append(step)
        if min(steps) != max(steps):
            raise ValueError("gate, gain and shift must have one stride between streams")
    r = Residual(_ptr(x), _ptr(o), _ptr(post_w), _ptr(pre_w), gp, ap, sp, step, res_scale)
    _check(load().bdssm_residual_norm(ctypes.byref(nd), ctypes.byref(r), _ptr(x_out), _ptr(u), _stream(stream)))


def attn_dims(batch, nheads, kv_heads, headdim, dtype, page_size):
    return AttnDims(batch, nheads, kv_heads, headdim, dtype, page_size)


def attn_mask(scale, block=0, window=0, sinks=0):
    """A bdssm_attn_mask: block 0 = no order, 1 = causal, n = by blocks of n; window 0 = none."""
    return AttnMask(scale, block, window, sinks)


class KvCache:
    """A paged cache as the attention calls take it: pools k, v [num_pages, kv_heads, page_size,
    headdim], table [batch, max_pages] int32 and lens [batch] int32, all on the device, and
    max_len, an upper bound of lens. Keeps the tensors whose addresses it holds; their contents
    may change between calls."""

    def __init__(self, ad, k, v, table, lens, max_len):
        import torch
        shape = (k.shape[0], ad.kv_heads, ad.page_size, ad.headdim)
        for t, what in ((k, "k"), (v, "v")):
            _expect(t, what, _torch_dtype(ad.dtype), shape)
        _expect(table, "table", torch.int32, (ad.batch, table.shape[-1]))
        _expect(lens, "lens", torch.int32, (ad.batch,))
        self.k, self.v, self.table, self.lens = k, v, table, lens
        self.page = (ad.kv_heads, ad.headdim, ad.page_size, ad.dtype)
        self.ptrs = KvCachePtrs(_ptr(k), _ptr(v), _ptr(table), _ptr(lens), k.shape[0], table.shape[1], max_len)

    @property
    def max_len(self):
        return self.ptrs.max_len

    @max_len.setter
    def max_len(self, n):
        self.ptrs.max_len = n

    def set_lens(self, lens):
        """Another lengths tensor (the lens_out of an append)."""
        import torch
        _expect(lens, "lens", torch.int32, self.lens.shape)
        self.ptrs.lens, self.lens = _ptr(lens), lens


def _chunk(ad, block_len, q, k, v, starts):
    """A bdssm_attn_chunk of q [tokens, nheads, headdim], k, v [tokens, kv_heads, headdim] (rows
    may be slices of longer ones) and starts [batch + 1] int32 or None."""
    dt, D, kv = _torch_dtype(ad.dtype), ad.headdim, ad.kv_heads
    n = (q if q is not None else k).shape[0]
    qp = kp = vp = sp = None
    qs = ks = vs = 0
    if q is not None:
        qp, qs = _rows(q, "q", dt, (n, ad.nheads, D))
    if k is not None:
        kp, ks = _rows(k, "k", dt, (n, kv, D))
    if v is not None:
        vp, vs = _rows(v, "v", dt, (n, kv, D))
    if starts is not None:
        import torch
        _expect(starts, "starts", torch.int32, (ad.batch + 1,))
        sp = _ptr(starts)
    return AttnChunk(qp, kp, vp, qs, ks, vs, n, sp, block_len)


def attn_step_workspace(ad, block_len, max_len, mask):
    """bdssm_attn_step_workspace: bytes that serve max_len and every smaller one (SIZE_MAX for
    arguments the call would reject)."""
    return load().bdssm_attn_step_workspace(ctypes.byref(ad), block_len, max_len, ctypes.byref(mask))


def attn_step(ad, block_len, q, k, v, cache, mask, out, workspace=None, starts=None, stream=None):
    """bdssm_attn_step: attention of the chunk's tokens over the cache and the chunk (k = v = None:
    over the cache alone); out [tokens, nheads, headdim] contiguous."""
    ch = _chunk(ad, block_len, q, k, v, starts)
    _expect(out, "out", q.dtype, q.shape)
    _check(load().bdssm_attn_step(ctypes.byref(ad), ctypes.byref(ch), ctypes.byref(cache.ptrs), ctypes.byref(mask),
                                  _ptr(out), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def kv_append(ad, block_len, k, v, cache, lens_out=None, starts=None, stream=None):
    """bdssm_kv_append: the chunk's keys and values into the cache's pages; lens_out [batch] int32
    receives the new lengths."""
    if lens_out is not None:
        _expect(lens_out, "lens_out", cache.lens.dtype, (ad.batch,))
    ch = _chunk(ad, block_len, None, k, v, starts)
    _check(load().bdssm_kv_append(ctypes.byref(ad), ctypes.byref(ch), ctypes.byref(cache.ptrs), _ptr(lens_out),
                                  _stream(stream)))


class AttnScores:
    """What bdssm_attn_step_ex does to the scores and the mask: cap (0 = none), slopes [nheads]
    float32 of the distance bias, prefix [batch] int32, and first, last [tokens] int32, the range of
    keys of every chunk row; all but cap on the device, each or None. Keeps the tensors whose
    addresses it holds; their contents may change between calls."""

    def __init__(self, cap=0.0, slopes=None, prefix=None, first=None, last=None):
        import torch
        for t, what, dtype in ((slopes, "slopes", torch.float32), (prefix, "prefix", torch.int32),
                               (first, "first", torch.int32), (last, "last", torch.int32)):
            if t is not None and t.dtype != dtype:
                raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
        self.slopes, self.prefix, self.first, self.last = slopes, prefix, first, last
        self.ptrs = AttnScoresPtrs(cap, _ptr(slopes), _ptr(prefix), _ptr(first), _ptr(last))


def attn_step_ex_workspace(ad, block_len, max_len, mask, scores):
    """bdssm_attn_step_ex_workspace: bytes that serve max_len and every smaller one (SIZE_MAX for
    arguments the call would reject)."""
    return load().bdssm_attn_step_ex_workspace(ctypes.byref(ad), block_len, max_len, ctypes.byref(mask),
                                               ctypes.byref(scores.ptrs))


def attn_step_ex(ad, block_len, q, k, v, cache, mask, scores, out, workspace=None, starts=None, stream=None):
    """bdssm_attn_step_ex: attn_step with the scores shaped and the rows' ranges limited by scores
    (an AttnScores)."""
    ch = _chunk(ad, block_len, q, k, v, starts)
    _expect(out, "out", q.dtype, q.shape)
    for t, what, n in ((scores.slopes, "slopes", ad.nheads), (scores.prefix, "prefix", ad.batch),
                       (scores.first, "first", ch.tokens), (scores.last, "last", ch.tokens)):
        if t is not None and t.shape != (n,):
            raise ValueError(f"{what}: expected ({n},), got {tuple(t.shape)}")
    _check(load().bdssm_attn_step_ex(ctypes.byref(ad), ctypes.byref(ch), ctypes.byref(cache.ptrs), ctypes.byref(mask),
                                     ctypes.byref(scores.ptrs), _ptr(out), _ptr(workspace), _nbytes(workspace),
                                     _stream(stream)))


def rotary_turns(dim, base=10000.0, kind=ROTARY_PLAIN, factor=1.0, trained=0, low=1.0, high=32.0, device="cuda"):
    """bdssm_rotary_turns: the frequencies of dim rotated channels as turns per position in units of
    2^-64, [dim / 2] int64 (the bits of uint64) on the device."""
    import torch
    out = np.zeros(max(dim // 2, 1), dtype=np.uint64)
    f = RotaryFreqs(dim, kind, base, factor, trained, low, high)
    _check(load().bdssm_rotary_turns(ctypes.byref(f), out.ctypes.data))
    return torch.from_numpy(out.view(np.int64)).to(device)


class Rotary:
    """A bdssm_rotary: turns (of rotary_turns; they say how many channels are rotated), the pairs'
    layout and the scale. positions [tokens] int32 replaces the cache's own positions (None). Keeps
    the tensors whose addresses it holds."""

    def __init__(self, turns, interleaved=False, scale=1.0, positions=None):
        import torch
        _expect(turns, "turns", torch.int64, (turns.numel(),))
        if positions is not None:
            _expect(positions, "positions", torch.int32, (positions.numel(),))
        self.turns, self.positions = turns, positions
        self.ptrs = RotaryPtrs(2 * turns.numel(), int(interleaved), scale, _ptr(turns), _ptr(positions))


def _rotary_out(ad, rotary, ch, q_out, k_out):
    if rotary.positions is not None and rotary.positions.shape != (ch.tokens,):
        raise ValueError(f"positions: expected ({ch.tokens},), got {tuple(rotary.positions.shape)}")
    qp = kp = None
    qs = ks = 0
    dt, D = _torch_dtype(ad.dtype), ad.headdim
    if q_out is not None:
        qp, qs = _rows(q_out, "q_out", dt, (ch.tokens, ad.nheads, D))
    if k_out is not None:
        kp, ks = _rows(k_out, "k_out", dt, (ch.tokens, ad.kv_heads, D))
    return RotaryOut(qp, kp, qs, ks)


def rotary_step(ad, block_len, rotary, q, k, q_out, k_out, lens=None, starts=None, stream=None):
    """bdssm_rotary_step: q [tokens, nheads, headdim] turned into q_out and k [tokens, kv_heads,
    headdim] into k_out (q, k or other rows; each pair may be None); lens [batch] int32 or None."""
    ch = _chunk(ad, block_len, q, k, None, starts)
    out = _rotary_out(ad, rotary, ch, q_out, k_out)
    if lens is not None:
        _expect_int(lens, "lens", (ad.batch,))
    _check(load().bdssm_rotary_step(ctypes.byref(ad), ctypes.byref(ch), ctypes.byref(rotary.ptrs), _ptr(lens),
                                    ctypes.byref(out), _stream(stream)))


def rotary_append(ad, block_len, rotary, q, k, v, cache, q_out, k_out=None, lens_out=None, starts=None, stream=None):
    """bdssm_rotary_append: q turned into q_out, k turned into the cache's pages (and k_out), v into
    the pages; lens_out [batch] int32 receives the new lengths. q = q_out = None: keys alone."""
    if lens_out is not None:
        _expect(lens_out, "lens_out", cache.lens.dtype, (ad.batch,))
    ch = _chunk(ad, block_len, q, k, v, starts)
    out = _rotary_out(ad, rotary, ch, q_out, k_out)
    _check(load().bdssm_rotary_append(ctypes.byref(ad), ctypes.byref(ch), ctypes.byref(cache.ptrs),
                                      ctypes.byref(rotary.ptrs), ctypes.byref(out), _ptr(lens_out), _stream(stream)))


def page_dims(batch, page_size, num_pages, max_pages):
    return PagesDims(batch, page_size, num_pages, max_pages)


class Pages:
    """A paged cache's bookkeeping as the pages_* calls take it: table [batch, max_pages], lens
    [batch] and uses [num_pages], int32 on the device. Keeps the tensors whose addresses it holds;
    their contents may change between calls."""

    def __init__(self, pd, table, lens, uses):
        import torch
        _expect(table, "table", torch.int32, (pd.batch, pd.max_pages))
        _expect(lens, "lens", torch.int32, (pd.batch,))
        _expect(uses, "uses", torch.int32, (pd.num_pages,))
        self.table, self.lens, self.uses = table, lens, uses
        self.pd, self.sizes = pd, (pd.batch, pd.max_pages, pd.num_pages)
        self.ptrs = PagesPtrs(_ptr(table), _ptr(lens), _ptr(uses))


def _pages_of(pd, pages):
    if pages.pd is not pd and pages.sizes != (pd.batch, pd.max_pages, pd.num_pages):
        raise ValueError(f"pages: made for (batch, max_pages, num_pages) {pages.sizes}")


def pages_workspace(pd):
    """bdssm_pages_workspace: bytes that serve each of the pages_* calls (SIZE_MAX for dims that they
    would reject)."""
    return load().bdssm_pages_workspace(ctypes.byref(pd))


def pages_advance(pd, pages, block_len, table_out, uses_out, lacking, workspace, window=0, sinks=0, starts=None,
                  stream=None):
    """bdssm_pages_advance: the pages of the next block_len tokens (or of starts) taken, those behind
    the window given back; table_out and uses_out may be the pages' own; lacking [1] int32."""
    _pages_of(pd, pages)
    b = pd.batch
    _expect_int(table_out, "table_out", (b, pd.max_pages))
    _expect_int(uses_out, "uses_out", (pd.num_pages,))
    _expect_int(lacking, "lacking", (1,))
    if starts is not None:
        _expect_int(starts, "starts", (b + 1,))
    _check(load().bdssm_pages_advance(ctypes.byref(pd), ctypes.byref(pages.ptrs), _ptr(starts), block_len, window, sinks,
                                      _ptr(table_out), _ptr(uses_out), _ptr(lacking), _ptr(workspace), _nbytes(workspace),
                                      _stream(stream)))


def pages_fork(pd, pages, parents, table_out, lens_out, uses_out, copies, lacking, workspace, stream=None):
    """bdssm_pages_fork: row b becomes the stream of row parents[b] ([batch] int32); copies [batch, 2]
    int32 receives the page copies to be made in every layer (pages_copy), lacking [1] int32."""
    _pages_of(pd, pages)
    b = pd.batch
    _expect_int(parents, "parents", (b,))
    _expect_int(table_out, "table_out", (b, pd.max_pages))
    _expect_int(lens_out, "lens_out", (b,))
    _expect_int(uses_out, "uses_out", (pd.num_pages,))
    _expect_int(copies, "copies", (b, 2))
    _expect_int(lacking, "lacking", (1,))
    _check(load().bdssm_pages_fork(ctypes.byref(pd), ctypes.byref(pages.ptrs), _ptr(parents), _ptr(table_out),
                                   _ptr(lens_out), _ptr(uses_out), _ptr(copies), _ptr(lacking), _ptr(workspace),
                                   _nbytes(workspace), _stream(stream)))


def pages_compact(pd, pages, table_out, uses_out, copies, live, workspace, stream=None):
    """bdssm_pages_compact: the used pages moved to the front of the pool; copies [num_pages // 2, 2]
    int32 receives the moves to be made in every layer (pages_copy), live [1] int32 their number."""
    _pages_of(pd, pages)
    n = pd.num_pages
    _expect_int(table_out, "table_out", (pd.batch, pd.max_pages))
    _expect_int(uses_out, "uses_out", (n,))
    _expect_int(copies, "copies", (n // 2, 2))
    _expect_int(live, "live", (1,))
    _check(load().bdssm_pages_compact(ctypes.byref(pd), ctypes.byref(pages.ptrs), _ptr(table_out), _ptr(uses_out),
                                      _ptr(copies), _ptr(live), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def pages_copy(ad, cache, copies, stream=None):
    """bdssm_pages_copy: the pages of copies [n, 2] int32 (source, destination) copied within one
    layer's pools (a KvCache)."""
    if cache.page != (ad.kv_heads, ad.headdim, ad.page_size, ad.dtype):
        raise ValueError(f"cache: its pages are of (kv_heads, headdim, page_size, dtype) {cache.page}")
    n = copies.shape[0]
    _expect_int(copies, "copies", (n, 2))
    _check(load().bdssm_pages_copy(ctypes.byref(ad), ctypes.byref(cache.ptrs), _ptr(copies), n, _stream(stream)))


# ------------------------------------------------------------------ data movement helpers
def to_device(arr, device="cuda"):
    """numpy input array (float32, or uint16 bfloat16 patterns) -> torch device tensor."""
    import torch
    a = np.ascontiguousarray(arr)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
    return torch.from_numpy(a).to(device)


def seq_to_device(seq, device="cuda"):
    """An inputs.Seq -> (x, dt, B, C) device tensors."""
    return tuple(to_device(a, device) for a in (seq.x, seq.dt, seq.B, seq.C))
