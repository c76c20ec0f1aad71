"""Python binding of libbsq.so: block-scaled quantization (MXFP8, NVFP4, MXFP4) and the
block-scaled GEMM with a fused bias + bf16 epilogue on GB300 (sm_103a).

The functions named like the C ABI (``bsq_quantize``, ``bsq_gemm``, ...) only marshal
arguments: torch tensors are passed as device pointers, the current torch stream as the
CUDA stream. ``quantize`` / ``gemm`` / ``linear`` add output allocation with torch (device
memory is the only thing torch provides here). Every step of the computation runs in the
library's CUDA kernels; there is no other implementation, and importing this package
raises if libbsq.so is missing.
"""
from __future__ import annotations

import array
import ctypes
import dataclasses
import importlib.machinery
import importlib.util
import os
import struct
import sysconfig
import warnings
from typing import NamedTuple, Optional, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# BSQ_LIBRARY=checked selects the checked build (device-side index checks, status
# BSQ_ERR_DEVICE_CHECK on a failed check); the default is the normal build
LIB_PATH = os.path.join(_HERE, "libbsq_checked.so" if os.environ.get("BSQ_LIBRARY") == "checked" else "libbsq.so")

MXFP8, NVFP4, MXFP4 = 1, 2, 3
FLAG_SRC_F32 = 0x100
FLAG_GLOBAL_GIVEN = 0x200
FLAG_STOCHASTIC = 0x400
FORMATS = {"mxfp8": MXFP8, "nvfp4": NVFP4, "mxfp4": MXFP4}

OK, ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_ARCH, ERR_LAUNCH, ERR_TIMEOUT, ERR_DEVICE_CHECK = 0, -1, -2, -3, -4, -5, -6, -7

if not os.path.exists(LIB_PATH):
    raise ImportError("%s is not built (run block_scaled_precision_bsq_gb300.build.build() "
                      "or __graft_entry__.build()); there is no fallback implementation" % os.path.basename(LIB_PATH))

_lib = ctypes.CDLL(LIB_PATH)
_i64, _vp, _int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
_lib.bsq_codes_bytes.restype = ctypes.c_size_t
_lib.bsq_codes_bytes.argtypes = [_int, _i64, _i64]
_lib.bsq_scales_bytes.restype = ctypes.c_size_t
_lib.bsq_scales_bytes.argtypes = [_int, _i64, _i64]
_lib.bsq_quantize.restype = _int
_lib.bsq_quantize.argtypes = [_int, _vp, _i64, _i64, _vp, _vp, _vp, _vp]
MAX_BATCH = 8
MAX_EXPERTS = 2048
NORM_RMS, NORM_LAYER = 1, 2
NORM_KINDS = {"rms": NORM_RMS, "layer": NORM_LAYER}
FLAG_PARAMS_F32 = 0x800
FLAG_POST_NORM = 0x1000
FLAG_IDS_I64 = 0x2000
GRAD_NORM_L2, GRAD_NORM_MAX = 1, 2


class QuantItem(ctypes.Structure):
    """bsq_quant_item of bsq.h."""
    _fields_ = [("src", _vp), ("rows", _i64), ("cols", _i64), ("codes", _vp), ("scales", _vp),
                ("global_scale", ctypes.POINTER(ctypes.c_float))]


class BlockNormArgs(ctypes.Structure):
    """bsq_block_norm_args of bsq.h."""
    _fields_ = [("kind", ctypes.c_int32), ("flags", ctypes.c_int32), ("rows", _i64), ("cols", _i64),
                ("gate_groups", _i64), ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("h", _vp), ("x", _vp), ("h_stride", _i64), ("x_stride", _i64),
                ("post_weight", _vp), ("post_bias", _vp), ("gate", _vp), ("pre_weight", _vp), ("pre_bias", _vp),
                ("x_out", _vp), ("y", _vp), ("stats", _vp)]


class BlockNormGradArgs(ctypes.Structure):
    """bsq_block_norm_grad_args of bsq.h."""
    _fields_ = [("kind", ctypes.c_int32), ("flags", ctypes.c_int32), ("rows", _i64), ("cols", _i64),
                ("gate_groups", _i64), ("residual_scale", ctypes.c_float), ("weight_offset", ctypes.c_float),
                ("dx_out", _vp), ("dy", _vp), ("x_out", _vp), ("h", _vp), ("dx_out_stride", _i64),
                ("dy_stride", _i64), ("x_out_stride", _i64), ("h_stride", _i64), ("stats", _vp),
                ("post_weight", _vp), ("post_bias", _vp), ("gate", _vp), ("pre_weight", _vp), ("pre_bias", _vp),
                ("dx", _vp), ("dh", _vp), ("dpost_weight", _vp), ("dpost_bias", _vp), ("dgate", _vp),
                ("dpre_weight", _vp), ("dpre_bias", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


# the same two as packed bytes: 1 us a call less than filling a Structure
_NORM_ARGS = struct.Struct("@iiqqqfffPPqqPPPPPPPP")
_NORM_GRAD_ARGS = struct.Struct("@iiqqqffPPPPqqqqPPPPPPPPPPPPPPN")
assert _NORM_ARGS.size == ctypes.sizeof(BlockNormArgs) and _NORM_GRAD_ARGS.size == ctypes.sizeof(BlockNormGradArgs)


class GradItem(ctypes.Structure):
    """bsq_grad_item of bsq.h."""
    _fields_ = [("src", _vp), ("dst", _vp), ("elems", _i64), ("f32", ctypes.c_int32)]


_lib.bsq_block_norm.restype = _int
_lib.bsq_block_norm.argtypes = [_vp, _vp]
_lib.bsq_block_norm_backward.restype = _int
_lib.bsq_block_norm_backward.argtypes = [_vp, _vp]
_lib.bsq_block_norm_backward_workspace.restype = ctypes.c_size_t
_lib.bsq_block_norm_backward_workspace.argtypes = [_int, _i64, _i64, _i64]
_lib.bsq_expert_sort.restype = _int
_lib.bsq_expert_sort.argtypes = [_int, _vp, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.bsq_expert_capacity.restype = _i64
_lib.bsq_expert_capacity.argtypes = [_i64, _i64, _i64]
_lib.bsq_expert_sort_workspace.restype = ctypes.c_size_t
_lib.bsq_expert_sort_workspace.argtypes = [_i64, _i64]
_lib.bsq_expert_gather.restype = _int
_lib.bsq_expert_gather.argtypes = [_int, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp]
_lib.bsq_expert_combine.restype = _int
_lib.bsq_expert_combine.argtypes = [_int, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp]
_lib.bsq_expert_combine_backward.restype = _int
_lib.bsq_expert_combine_backward.argtypes = [_int, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp,
                                             _vp]
_lib.bsq_grad_norm.restype = _int
_lib.bsq_grad_norm.argtypes = [_int, ctypes.POINTER(GradItem), _int, _vp, _vp, ctypes.c_size_t, _vp]
_lib.bsq_clip_grad_norm.restype = _int
_lib.bsq_clip_grad_norm.argtypes = [_int, ctypes.POINTER(GradItem), _int, ctypes.c_float, ctypes.c_float, _vp, _vp,
                                    ctypes.c_size_t, _vp]
_lib.bsq_clip_grad_norm_workspace.restype = ctypes.c_size_t
_lib.bsq_clip_grad_norm_workspace.argtypes = [_int]
_lib.bsq_quantize_batch.restype = _int
_lib.bsq_quantize_batch.argtypes = [_int, _int, ctypes.POINTER(QuantItem), _vp]
_lib.bsq_layernorm_quantize.restype = _int
_lib.bsq_layernorm_quantize.argtypes = [_int, _vp, _vp, _vp, ctypes.c_float, _i64, _i64, _vp, _vp, _vp]
_lib.bsq_gemm.restype = _int
_lib.bsq_quantize_dual.argtypes = [_int, _vp, _i64, _i64, ctypes.c_uint64, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.bsq_quantize_dual.restype = _int
_lib.bsq_delayed_global_scale.argtypes = [_vp, _i64, _i64, ctypes.c_float, _vp, _vp]
_lib.bsq_delayed_global_scale.restype = _int
_lib.bsq_convt2x2.argtypes = [_int, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _int, _vp]
_lib.bsq_convt2x2.restype = _int
_lib.bsq_gemm.argtypes = [_int, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp]
_lib.bsq_gemm_splitk.restype = _int
_lib.bsq_gemm_splitk.argtypes = [_int, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, ctypes.c_size_t, _vp]
_lib.bsq_gemm_splitk_scratch.restype = _int
_lib.bsq_gemm_splitk_scratch.argtypes = [_int, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp]
_lib.bsq_gemm_splitk_splits.restype = _int
_lib.bsq_gemm_splitk_splits.argtypes = [_int, _i64, _i64, _i64]
_lib.bsq_gemm_gelu.restype = _int
_lib.bsq_gemm_gelu.argtypes = [_int, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp]
_lib.bsq_gemm_gelu_quantize.restype = _int
_lib.bsq_gemm_gelu_quantize.argtypes = [_int, _vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _i64, _i64, _i64, _vp]
_lib.bsq_get_device_status.restype = _int
_lib.bsq_get_device_status.argtypes = [_vp]
_lib.bsq_selftest_timeout.restype = _int
_lib.bsq_selftest_timeout.argtypes = [_i64, _vp]
_lib.bsq_selftest_device_check.restype = _int
_lib.bsq_selftest_device_check.argtypes = [_vp]
_lib.bsq_test_inject_stall.restype = _int
_lib.bsq_test_inject_stall.argtypes = [_int, _i64, _i64]
KERNEL_GEMM, KERNEL_DUAL, KERNEL_LAYERNORM, KERNEL_NORM = 1, 2, 3, 5
_lib.bsq_test_norm_cut.restype = _int
_lib.bsq_test_norm_cut.argtypes = [_int, _i64, _i64, _i64, _i64, _int, _int, ctypes.POINTER(_i64)]
_lib.bsq_last_error.restype = _int
_lib.bsq_strerror.restype = ctypes.c_char_p
_lib.bsq_strerror.argtypes = [_int]

EXPORTS = ("bsq_codes_bytes", "bsq_scales_bytes", "bsq_quantize", "bsq_quantize_batch", "bsq_layernorm_quantize",
           "bsq_quantize_dual", "bsq_delayed_global_scale", "bsq_gemm", "bsq_gemm_splitk", "bsq_gemm_splitk_splits",
           "bsq_gemm_splitk_scratch",
           "bsq_gemm_gelu", "bsq_gemm_gelu_quantize", "bsq_convt2x2", "bsq_block_norm", "bsq_block_norm_backward",
           "bsq_block_norm_backward_workspace", "bsq_expert_sort", "bsq_expert_capacity", "bsq_expert_sort_workspace",
           "bsq_expert_gather", "bsq_expert_combine", "bsq_expert_combine_backward", "bsq_grad_norm",
           "bsq_clip_grad_norm", "bsq_clip_grad_norm_workspace", "bsq_get_device_status", "bsq_selftest_timeout",
           "bsq_selftest_device_check", "bsq_test_inject_stall", "bsq_test_norm_cut",
           "bsq_last_error", "bsq_strerror")



_FAST_CALLS = ("bsq_block_norm", "bsq_block_norm_backward", "bsq_block_norm_backward_workspace", "bsq_expert_sort",
               "bsq_expert_capacity", "bsq_expert_sort_workspace", "bsq_expert_gather", "bsq_expert_combine",
               "bsq_expert_combine_backward", "bsq_grad_norm", "bsq_clip_grad_norm", "bsq_clip_grad_norm_workspace")


def _binding_stamp() -> str:
    """What _bsq_torch.so was built against: this torch, under this Python."""
    return "%s %s" % (torch.__version__, sysconfig.get_config_var("SOABI"))


def _load_fast():
    """The host side of the functions around the linear layers in C++ (csrc/bsq_torch.cpp), or None
    where it was not built for this torch and Python or does not load. The same library calls either way."""
    path = os.path.join(_HERE, "_bsq_torch.so")
    if not os.path.exists(path):
        return None
    try:
        with open(path + ".torch") as f:
            if f.read() != _binding_stamp():
                return None
    except OSError:
        return None
    try:
        loader = importlib.machinery.ExtensionFileLoader("_bsq_torch", path)
        spec = importlib.util.spec_from_file_location("_bsq_torch", path, loader=loader)
        mod = importlib.util.module_from_spec(spec)
        loader.exec_module(mod)
        mod.init(*(ctypes.cast(getattr(_lib, n), _vp).value for n in _FAST_CALLS))
    except (ImportError, TypeError) as e:  # TypeError: built from an older list of functions
        warnings.warn("_bsq_torch.so is not used: %s" % e, RuntimeWarning)
        return None
    return mod


_fast = _load_fast()

Ptr = Union[int, None, torch.Tensor]


class BsqError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__("%s failed: %d (%s)" % (what, code, bsq_strerror(code)))
        self.code = code


def _p(x: Ptr) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        return x.data_ptr() if x.numel() > 0 else None
    return int(x)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _current_stream() -> Optional[int]:
    """The current stream's handle. torch.cuda.current_stream() makes a Stream object each time, which
    costs more than the launch (5.5 us of a 12 us call); the handle alone takes 0.1 us."""
    if not torch.cuda.is_initialized() and not torch.cuda.is_available():  # the latter asks the driver each time
        return None
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


# ---------------------------------------------------------------- C ABI, one to one
def bsq_codes_bytes(fmt, rows: int, cols: int) -> int:
    return int(_lib.bsq_codes_bytes(_fmt(fmt), rows, cols))


def bsq_scales_bytes(fmt, rows: int, cols: int) -> int:
    return int(_lib.bsq_scales_bytes(_fmt(fmt), rows, cols))


def bsq_quantize(fmt_flags: int, src: Ptr, rows: int, cols: int, codes: Ptr, scales: Ptr,
                 global_scale: Ptr = None, stream=None) -> int:
    return int(_lib.bsq_quantize(int(fmt_flags), _p(src), rows, cols, _p(codes), _p(scales), _p(global_scale),
                                 _stream(stream)))


def bsq_quantize_batch(fmt_flags: int, items, stream=None) -> int:
    """items: sequence of (src, rows, cols, codes, scales, global_scale) tuples (pointers or
    tensors, as bsq_quantize takes them)."""
    arr = (QuantItem * max(1, len(items)))()
    for i, (src, rows, cols, codes, scales, gs) in enumerate(items):
        g = _p(gs)
        arr[i] = QuantItem(_p(src), rows, cols, _p(codes), _p(scales),
                           ctypes.cast(g, ctypes.POINTER(ctypes.c_float)) if g else None)
    return int(_lib.bsq_quantize_batch(int(fmt_flags), len(items), arr, _stream(stream)))


def bsq_layernorm_quantize(fmt_flags: int, src: Ptr, gamma: Ptr, beta: Ptr, eps: float, rows: int, cols: int,
                           codes: Ptr, scales: Ptr, stream=None) -> int:
    return int(_lib.bsq_layernorm_quantize(int(fmt_flags), _p(src), _p(gamma), _p(beta), float(eps), rows, cols,
                                           _p(codes), _p(scales), _stream(stream)))


def bsq_quantize_dual(fmt_flags: int, src: Ptr, rows: int, cols: int, seed: int, row_codes: Ptr, row_scales: Ptr,
                      col_codes: Ptr, col_scales: Ptr, global_scale: Ptr = None, stream=None) -> int:
    return int(_lib.bsq_quantize_dual(int(fmt_flags), _p(src), rows, cols, int(seed) & (2 ** 64 - 1), _p(row_codes),
                                      _p(row_scales), _p(col_codes), _p(col_scales), _p(global_scale),
                                      _stream(stream)))


def bsq_delayed_global_scale(prev_scales: Ptr, rows: int, cols: int, headroom: float, g_out: Ptr,
                             stream=None) -> int:
    return int(_lib.bsq_delayed_global_scale(_p(prev_scales), rows, cols, float(headroom), _p(g_out),
                                             _stream(stream)))


def bsq_gemm(fmt, A: Ptr, A_scales: Ptr, B: Ptr, B_scales: Ptr, bias: Ptr, out: Ptr, M: int, N: int, K: int,
             stream=None) -> int:
    return int(_lib.bsq_gemm(_fmt(fmt), _p(A), _p(A_scales), _p(B), _p(B_scales), _p(bias), _p(out), M, N, K,
                             _stream(stream)))


def bsq_gemm_splitk(fmt, A: Ptr, A_scales: Ptr, B: Ptr, B_scales: Ptr, bias: Ptr, out: Ptr, M: int, N: int, K: int,
                    splits: int, workspace: Ptr, workspace_bytes: int, stream=None) -> int:
    return int(_lib.bsq_gemm_splitk(_fmt(fmt), _p(A), _p(A_scales), _p(B), _p(B_scales), _p(bias), _p(out), M, N, K,
                                    splits, _p(workspace), workspace_bytes, _stream(stream)))


def bsq_gemm_splitk_scratch(fmt, A: Ptr, A_scales: Ptr, B: Ptr, B_scales: Ptr, bias: Ptr, out: Ptr, M: int, N: int,
                            K: int, splits: int, stream=None) -> int:
    return int(_lib.bsq_gemm_splitk_scratch(_fmt(fmt), _p(A), _p(A_scales), _p(B), _p(B_scales), _p(bias), _p(out),
                                            M, N, K, splits, _stream(stream)))


def bsq_gemm_splitk_splits(fmt, M: int, N: int, K: int) -> int:
    return int(_lib.bsq_gemm_splitk_splits(_fmt(fmt), M, N, K))


def bsq_gemm_gelu(fmt, A: Ptr, A_scales: Ptr, B: Ptr, B_scales: Ptr, bias: Ptr, out: Ptr, M: int, N: int,
                  K: int, stream=None) -> int:
    return int(_lib.bsq_gemm_gelu(_fmt(fmt), _p(A), _p(A_scales), _p(B), _p(B_scales), _p(bias), _p(out), M, N, K,
                                  _stream(stream)))


def bsq_gemm_gelu_quantize(fmt, A: Ptr, A_scales: Ptr, B: Ptr, B_scales: Ptr, bias: Ptr, out_fmt, out_codes: Ptr,
                           out_scales: Ptr, M: int, N: int, K: int, stream=None) -> int:
    return int(_lib.bsq_gemm_gelu_quantize(_fmt(fmt), _p(A), _p(A_scales), _p(B), _p(B_scales), _p(bias),
                                           _fmt(out_fmt), _p(out_codes), _p(out_scales), M, N, K, _stream(stream)))


def bsq_convt2x2(fmt, A: Ptr, A_scales: Ptr, B: Ptr, B_scales: Ptr, bias: Ptr, out: Ptr, batch: int, H: int, W: int,
                 C_in: int, C_out: int, gelu: bool = False, stream=None) -> int:
    return int(_lib.bsq_convt2x2(_fmt(fmt), _p(A), _p(A_scales), _p(B), _p(B_scales), _p(bias), _p(out), batch, H, W,
                                 C_in, C_out, 1 if gelu else 0, _stream(stream)))


def bsq_block_norm(args: BlockNormArgs, stream=None) -> int:
    return int(_lib.bsq_block_norm(ctypes.byref(args), _stream(stream)))


def bsq_block_norm_backward(args: BlockNormGradArgs, stream=None) -> int:
    return int(_lib.bsq_block_norm_backward(ctypes.byref(args), _stream(stream)))


def bsq_block_norm_backward_workspace(flags: int, rows: int, cols: int, gate_groups: int = 1) -> int:
    return int(_lib.bsq_block_norm_backward_workspace(int(flags), rows, cols, gate_groups))


def bsq_expert_sort(flags: int, ids: Ptr, tokens: int, topk: int, experts: int, align: int, capacity: int, counts: Ptr,
                    offsets: Ptr, position: Ptr, slot: Ptr, workspace: Ptr = None, workspace_bytes: int = 0,
                    stream=None) -> int:
    return int(_lib.bsq_expert_sort(int(flags), _p(ids), tokens, topk, experts, align, capacity, _p(counts),
                                    _p(offsets), _p(position), _p(slot), _p(workspace), workspace_bytes,
                                    _stream(stream)))


def bsq_expert_capacity(slots: int, experts: int, align: int = 1) -> int:
    return int(_lib.bsq_expert_capacity(slots, experts, align))


def bsq_expert_sort_workspace(slots: int, experts: int) -> int:
    return int(_lib.bsq_expert_sort_workspace(slots, experts))


def bsq_expert_gather(flags: int, x: Ptr, x_stride: int, position: Ptr, slot: Ptr, tokens: int, topk: int, cols: int,
                      capacity: int, rows: Ptr, stream=None) -> int:
    return int(_lib.bsq_expert_gather(int(flags), _p(x), x_stride, _p(position), _p(slot), tokens, topk, cols, capacity,
                                      _p(rows), _stream(stream)))


def bsq_expert_combine(flags: int, y: Ptr, y_stride: int, position: Ptr, weights: Ptr, tokens: int, topk: int,
                       cols: int, capacity: int, out: Ptr, stream=None) -> int:
    return int(_lib.bsq_expert_combine(int(flags), _p(y), y_stride, _p(position), _p(weights), tokens, topk, cols,
                                       capacity, _p(out), _stream(stream)))


def bsq_expert_combine_backward(flags: int, dout: Ptr, dout_stride: int, y: Ptr, y_stride: int, position: Ptr,
                                slot: Ptr, weights: Ptr, tokens: int, topk: int, cols: int, capacity: int, dy: Ptr,
                                dweights: Ptr, stream=None) -> int:
    return int(_lib.bsq_expert_combine_backward(int(flags), _p(dout), dout_stride, _p(y), y_stride, _p(position),
                                                _p(slot), _p(weights), tokens, topk, cols, capacity, _p(dy),
                                                _p(dweights), _stream(stream)))


def _grad_items(items):
    """items: a ctypes array of GradItem, or a sequence of (src, dst, elems, f32) tuples (pointers or tensors)."""
    if isinstance(items, ctypes.Array):
        return len(items), items
    arr = (GradItem * max(1, len(items)))()
    for i, (src, dst, elems, f32) in enumerate(items):
        arr[i] = GradItem(_p(src), _p(dst), elems, 1 if f32 else 0)
    return len(items), arr


def bsq_grad_norm(items, norm_kind: int, norm: Ptr, workspace: Ptr, workspace_bytes: int, stream=None) -> int:
    n, arr = _grad_items(items)
    return int(_lib.bsq_grad_norm(n, arr, int(norm_kind), _p(norm), _p(workspace), workspace_bytes, _stream(stream)))


def bsq_clip_grad_norm(items, norm_kind: int, max_norm: float, eps: float, norm: Ptr, workspace: Ptr,
                       workspace_bytes: int, stream=None) -> int:
    n, arr = _grad_items(items)
    return int(_lib.bsq_clip_grad_norm(n, arr, int(norm_kind), float(max_norm), float(eps), _p(norm), _p(workspace),
                                       workspace_bytes, _stream(stream)))


def bsq_clip_grad_norm_workspace(count: int) -> int:
    return int(_lib.bsq_clip_grad_norm_workspace(int(count)))


def bsq_get_device_status(stream=None) -> int:
    return int(_lib.bsq_get_device_status(_stream(stream)))


def bsq_selftest_timeout(limit_ns: int, stream=None) -> int:
    return int(_lib.bsq_selftest_timeout(int(limit_ns), _stream(stream)))


def bsq_selftest_device_check(stream=None) -> int:
    return int(_lib.bsq_selftest_device_check(_stream(stream)))


class NormCut(NamedTuple):
    """bsq_test_norm_cut's answer."""
    vectors: int
    cluster: int
    warps: int
    teams: int
    classes: int
    rows_per_block: int
    blocks: int
    workspace: int


def bsq_test_norm_cut(flags: int, rows: int, cols: int, gate_groups: int = 1, widest: int = 0, vectors: bool = True,
                      num_sms: int = 152) -> NormCut:
    cut = (_i64 * 8)()
    rc = int(_lib.bsq_test_norm_cut(int(flags), rows, cols, gate_groups, widest, 1 if vectors else 0, num_sms, cut))
    if rc != OK:
        raise BsqError(rc, "bsq_test_norm_cut")
    return NormCut(*cut)


def bsq_test_inject_stall(kernel: int, after_stages: int, wait_limit_ns: int) -> int:
    return int(_lib.bsq_test_inject_stall(int(kernel), int(after_stages), int(wait_limit_ns)))


def bsq_last_error() -> int:
    return int(_lib.bsq_last_error())


def bsq_strerror(code: int) -> str:
    return _lib.bsq_strerror(int(code)).decode()


# ---------------------------------------------------------------- tensor-level helpers
@dataclasses.dataclass
class QTensor:
    """A quantized rows x cols matrix: packed codes, tiled scales (with the NVFP4 tail) and,
    for NVFP4, a one-element fp32 tensor holding the per-tensor scale g."""

    fmt: int
    rows: int
    cols: int
    codes: torch.Tensor
    scales: torch.Tensor
    global_scale: Optional[torch.Tensor] = None


def empty_qtensor(fmt, rows: int, cols: int, device="cuda") -> QTensor:
    f = _fmt(fmt)
    codes = torch.empty(bsq_codes_bytes(f, rows, cols), dtype=torch.uint8, device=device)
    scales = torch.empty(bsq_scales_bytes(f, rows, cols), dtype=torch.uint8, device=device)
    g = torch.empty(1, dtype=torch.float32, device=device) if f == NVFP4 else None
    return QTensor(f, rows, cols, codes, scales, g)


def _on_current_device(*tensors: Optional[torch.Tensor]) -> None:
    """The library launches on the current device: no tensor may lie on another."""
    here = torch.cuda.current_device()
    for t in tensors:
        assert t is None or t.get_device() == here, "all tensors must be on the current device"


def quantize(fmt, x: torch.Tensor, global_scale: Optional[torch.Tensor] = None, out: Optional[QTensor] = None,
             stream=None) -> QTensor:
    """Quantize a contiguous bf16 or fp32 CUDA matrix along its last dimension."""
    f = _fmt(fmt)
    assert x.is_cuda and x.is_contiguous() and x.dim() == 2, "x must be a contiguous 2-D CUDA tensor"
    rows, cols = x.shape
    flags = f
    if x.dtype == torch.float32:
        flags |= FLAG_SRC_F32
    elif x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16 or float32")
    q = out if out is not None else empty_qtensor(f, rows, cols, x.device)
    g = q.global_scale
    if global_scale is not None:
        flags |= FLAG_GLOBAL_GIVEN
        g = global_scale
    _on_current_device(x, q.codes, q.scales, g)
    rc = bsq_quantize(flags, x, rows, cols, q.codes, q.scales, g, stream)
    if rc != OK:
        raise BsqError(rc, "bsq_quantize")
    if global_scale is not None:
        q.global_scale = global_scale
    return q


def quantize_many(fmt, xs, outs=None, stream=None):
    """Quantize several contiguous 2-D CUDA matrices of one dtype (bf16 or fp32) in one launch
    (bsq_quantize_batch); NVFP4 computes each matrix's own g. Returns a list of QTensor."""
    f = _fmt(fmt)
    assert 1 <= len(xs) <= MAX_BATCH, "1..%d matrices per call" % MAX_BATCH
    dt = xs[0].dtype
    for x in xs:
        assert x.is_cuda and x.is_contiguous() and x.dim() == 2 and x.dtype == dt, \
            "matrices must be contiguous 2-D CUDA tensors of one dtype"
    flags = f
    if dt == torch.float32:
        flags |= FLAG_SRC_F32
    elif dt != torch.bfloat16:
        raise TypeError("matrices must be bfloat16 or float32")
    qs = list(outs) if outs is not None else [empty_qtensor(f, x.shape[0], x.shape[1], x.device) for x in xs]
    items = [(x, x.shape[0], x.shape[1], q.codes, q.scales, q.global_scale) for x, q in zip(xs, qs)]
    for x, q in zip(xs, qs):
        _on_current_device(x, q.codes, q.scales, q.global_scale)
    rc = bsq_quantize_batch(flags, items, stream)
    if rc != OK:
        raise BsqError(rc, "bsq_quantize_batch")
    return qs


def layernorm_quantize(fmt, x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float = 1e-6,
                       out: Optional[QTensor] = None, stream=None) -> QTensor:
    """Row LayerNorm (gamma, beta bf16) of a contiguous bf16 / fp32 CUDA matrix, quantized along
    the row into MXFP8 / MXFP4 in the same kernel."""
    f = _fmt(fmt)
    assert x.is_cuda and x.is_contiguous() and x.dim() == 2, "x must be a contiguous 2-D CUDA tensor"
    rows, cols = x.shape
    assert gamma.dtype == torch.bfloat16 and beta.dtype == torch.bfloat16 and gamma.numel() == cols == beta.numel()
    flags = f | (FLAG_SRC_F32 if x.dtype == torch.float32 else 0)
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("x must be bfloat16 or float32")
    q = out if out is not None else empty_qtensor(f, rows, cols, x.device)
    _on_current_device(x, gamma, beta, q.codes, q.scales)
    rc = bsq_layernorm_quantize(flags, x, gamma, beta, eps, rows, cols, q.codes, q.scales, stream)
    if rc != OK:
        raise BsqError(rc, "bsq_layernorm_quantize")
    return q


def quantize_dual(fmt, x: torch.Tensor, stochastic: bool = False, seed: int = 0,
                  global_scale: Optional[torch.Tensor] = None, out=None, stream=None):
    """Both operands of a contiguous bf16 / fp32 CUDA matrix X (R x C, multiples of 32) in one
    launch: (row-wise QTensor R x C, column-wise QTensor C x R = X^T quantized along R), with
    round-to-nearest-even or Philox-keyed stochastic rounding. NVFP4 shares one per-tensor
    scale between the layouts: computed from X, or `global_scale` (a one-element fp32 tensor)."""
    f = _fmt(fmt)
    assert x.is_cuda and x.is_contiguous() and x.dim() == 2, "x must be a contiguous 2-D CUDA tensor"
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("x must be bfloat16 or float32")
    rows, cols = x.shape
    flags = f | (FLAG_SRC_F32 if x.dtype == torch.float32 else 0) | (FLAG_STOCHASTIC if stochastic else 0)
    qr, qc = out if out is not None else (empty_qtensor(f, rows, cols, x.device), empty_qtensor(f, cols, rows, x.device))
    g = qr.global_scale
    if global_scale is not None:
        flags |= FLAG_GLOBAL_GIVEN
        g = global_scale
    _on_current_device(x, qr.codes, qr.scales, qc.codes, qc.scales, g)
    rc = bsq_quantize_dual(flags, x, rows, cols, seed, qr.codes, qr.scales, qc.codes, qc.scales, g, stream)
    if rc != OK:
        raise BsqError(rc, "bsq_quantize_dual")
    if f == NVFP4:
        qr.global_scale = g
        qc.global_scale = g
    return qr, qc


def delayed_global_scale(prev: QTensor, headroom: float = 32.0, out: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """The next step's NVFP4 per-tensor scale from an earlier quantization `prev` of the tensor:
    fp32(fp32(amax * headroom) / 2688) on the device, as a one-element fp32 tensor to pass as
    `global_scale`."""
    assert prev.fmt == NVFP4
    g = out if out is not None else torch.empty(1, dtype=torch.float32, device=prev.scales.device)
    _on_current_device(prev.codes, prev.scales, prev.global_scale, g)
    rc = bsq_delayed_global_scale(prev.scales, prev.rows, prev.cols, headroom, g, stream)
    if rc != OK:
        raise BsqError(rc, "bsq_delayed_global_scale")
    return g


def gemm(qa: QTensor, qb: QTensor, bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
         stream=None) -> torch.Tensor:
    """out[M, N] = bf16(alpha * A_hat . B_hat^T + bias), A: M x K, B: N x K (weight layout)."""
    assert qa.fmt == qb.fmt and qa.cols == qb.cols
    M, K, N = qa.rows, qa.cols, qb.rows
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=qa.codes.device)
    if bias is not None:
        assert bias.dtype == torch.bfloat16 and bias.numel() == N and bias.is_contiguous()
    _on_current_device(qa.codes, qa.scales, qb.codes, qb.scales, bias, out)
    rc = bsq_gemm(qa.fmt, qa.codes, qa.scales, qb.codes, qb.scales, bias, out, M, N, K, stream)
    if rc != OK:
        raise BsqError(rc, "bsq_gemm")
    return out


def gemm_splitk(qa: QTensor, qb: QTensor, bias: Optional[torch.Tensor] = None, splits: Optional[int] = None,
                workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """gemm() with K cut into `splits` ranges (default: the library's choice for the shape), the
    fp32 partial sums in `workspace` (splits x M x N fp32; allocated here when not given)."""
    assert qa.fmt == qb.fmt and qa.cols == qb.cols
    M, K, N = qa.rows, qa.cols, qb.rows
    if splits is None:
        splits = bsq_gemm_splitk_splits(qa.fmt, M, N, K)
        if splits < 0:
            raise BsqError(splits, "bsq_gemm_splitk_splits")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=qa.codes.device)
    if bias is not None:
        assert bias.dtype == torch.bfloat16 and bias.numel() == N and bias.is_contiguous()
    if workspace is None and splits > 1:
        workspace = torch.empty(splits * M * N, dtype=torch.float32, device=qa.codes.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _on_current_device(qa.codes, qa.scales, qb.codes, qb.scales, bias, workspace, out)
    rc = bsq_gemm_splitk(qa.fmt, qa.codes, qa.scales, qb.codes, qb.scales, bias, out, M, N, K, splits, workspace,
                         ws_bytes, stream)
    if rc != OK:
        raise BsqError(rc, "bsq_gemm_splitk")
    return out


def gemm_gelu(qa: QTensor, qb: QTensor, bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """out[M, N] = bf16(GELU(alpha * A_hat . B_hat^T + bias)), GELU in its erf form."""
    assert qa.fmt == qb.fmt and qa.cols == qb.cols
    M, K, N = qa.rows, qa.cols, qb.rows
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=qa.codes.device)
    _on_current_device(qa.codes, qa.scales, qb.codes, qb.scales, bias, out)
    rc = bsq_gemm_gelu(qa.fmt, qa.codes, qa.scales, qb.codes, qb.scales, bias, out, M, N, K, stream)
    if rc != OK:
        raise BsqError(rc, "bsq_gemm_gelu")
    return out


def gemm_gelu_quantize(qa: QTensor, qb: QTensor, bias: Optional[torch.Tensor] = None, out_fmt="mxfp8",
                       out: Optional[QTensor] = None, stream=None) -> QTensor:
    """GELU(alpha * A_hat . B_hat^T + bias) quantized along N into out_fmt (MXFP8 / MXFP4) in the
    GEMM's epilogue: an M x N operand, laid out as quantize() lays it out."""
    assert qa.fmt == qb.fmt and qa.cols == qb.cols
    M, K, N = qa.rows, qa.cols, qb.rows
    of = _fmt(out_fmt)
    q = out if out is not None else empty_qtensor(of, M, N, qa.codes.device)
    _on_current_device(qa.codes, qa.scales, qb.codes, qb.scales, bias, q.codes, q.scales)
    rc = bsq_gemm_gelu_quantize(qa.fmt, qa.codes, qa.scales, qb.codes, qb.scales, bias, of, q.codes, q.scales,
                                M, N, K, stream)
    if rc != OK:
        raise BsqError(rc, "bsq_gemm_gelu_quantize")
    return q


def linear(fmt, x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The whole block-scaled linear layer: quantize x and w along K, then the GEMM."""
    return gemm(quantize(fmt, x, stream=stream), quantize(fmt, w, stream=stream), bias, stream=stream)


def linear_backward(dy: torch.Tensor, x_col: QTensor, w_col: QTensor, stochastic: bool = False, seed: int = 0,
                    stream=None):
    """The two backward GEMMs of a block-scaled linear layer: dY (M x N, bf16 / fp32) is
    quantized in both layouts in one pass, then dX = dY . W (dY row-wise against W column-wise,
    M x K) and dW = dY^T . X (dY column-wise against X column-wise, N x K), both bf16 with fp32
    accumulation. x_col / w_col are the column-wise operands of X (M x K) and W (N x K) from
    quantize_dual (K x M and K x N). dW (few output tiles, K = the token count) goes through
    gemm_splitk with the library's split count. Returns (dX, dW)."""
    dy_row, dy_col = quantize_dual(x_col.fmt, dy, stochastic=stochastic, seed=seed, stream=stream)
    return gemm(dy_row, w_col, stream=stream), gemm_splitk(dy_col, x_col, stream=stream)


def convt2x2(qx: QTensor, qw: QTensor, batch: int, H: int, W: int, bias: Optional[torch.Tensor] = None,
             gelu: bool = False, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Kernel-2 stride-2 transposed convolution of a quantized NHWC input (batch*H*W x C_in) with a
    quantized 4*C_out x C_in weight (row (2 dy + dx) C_out + co): batch x 2H x 2W x C_out bf16."""
    assert qx.fmt == qw.fmt and qx.cols == qw.cols and qx.rows == batch * H * W and qw.rows % 4 == 0
    C_in, C_out = qx.cols, qw.rows // 4
    if out is None:
        out = torch.empty((batch, 2 * H, 2 * W, C_out), dtype=torch.bfloat16, device=qx.codes.device)
    _on_current_device(qx.codes, qx.scales, qw.codes, qw.scales, bias, out)
    rc = bsq_convt2x2(qx.fmt, qx.codes, qx.scales, qw.codes, qw.scales, bias, out, batch, H, W, C_in, C_out, gelu,
                      stream)
    if rc != OK:
        raise BsqError(rc, "bsq_convt2x2")
    return out


# ---------------------------------------------------------------- around the linear layers
# Small calls are bound by the host. A plain call goes through the C++ host side (_fast), which gives None
# for one that it does not take; the Python code below it does the same work, says what is wrong with the
# arguments, and serves where _fast is missing. An error code from _fast is a launch that failed behind others
# that may have run: it is raised, not tried again. All tensors of a call lie on the current device.
_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def _torch_stream(stream):
    """The stream of a call's `stream` argument: a torch stream or a handle. Handle 0 is the default
    stream: ExternalStream(0) would be a stream of torch's pool, which is ordered with nothing."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(stream)
    return torch.cuda.ExternalStream(handle) if handle != 0 else torch.cuda.default_stream()


def _taken(r, what: str):
    """What _fast returned for a call that it took."""
    if type(r) is int:
        raise BsqError(r, what)
    return r


def _addr(x: Optional[torch.Tensor]) -> int:
    return 0 if x is None else x.data_ptr()


def _handle(x: torch.Tensor) -> int:
    """The current stream of x's device."""
    return torch._C._cuda_getCurrentRawStream(x.get_device())


def _matrix(x: torch.Tensor, what: str, dtype=None, shape=None) -> int:
    """Checks a bf16 / fp32 CUDA matrix with unit column stride; returns its row stride."""
    dt = x.dtype
    if dt is not _BF16 and dt is not _F32 or dtype is not None and dt is not dtype:
        raise TypeError("%s must be %s" % (what, dtype if dtype is not None else "bfloat16 or float32"))
    strides = x.stride()
    assert x.is_cuda and len(strides) == 2 and (strides[1] == 1 or x.shape[1] == 1), \
        "%s must be a 2-D CUDA tensor with consecutive columns" % what
    assert shape is None or x.shape == shape, "%s has shape %s, not %s" % (what, tuple(x.shape), tuple(shape))
    return strides[0]


def _params(cols: int, gate, named) -> tuple:
    """Checks weights and biases (named) and gate: contiguous, one dtype. Returns (flag, gate groups)."""
    dtype, groups = None, 1
    if gate is not None:
        dtype, shape = gate.dtype, gate.shape
        if dtype is not _BF16 and dtype is not _F32:
            raise TypeError("gate must be bfloat16 or float32")
        assert gate.is_cuda and gate.is_contiguous(), "gate must be a contiguous CUDA tensor"
        assert len(shape) in (1, 2) and shape[-1] == cols, "gate must be cols or groups x cols"
        if len(shape) == 2:
            groups = shape[0]
            assert groups > 0, "gate must have a row"
    for name, p in named:
        if p is None:
            continue
        dt = p.dtype
        if dtype is None:
            dtype = dt
            if dt is not _BF16 and dt is not _F32:
                raise TypeError("%s must be bfloat16 or float32" % name)
        elif dt is not dtype:
            raise TypeError("weights, biases and gate must have one dtype")
        assert p.is_cuda and p.is_contiguous() and p.shape == (cols,), \
            "%s must be a contiguous CUDA tensor of %d values" % (name, cols)
    return (FLAG_PARAMS_F32 if dtype is _F32 else 0), groups


class BlockNorm(NamedTuple):
    x_out: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    stats: torch.Tensor


class BlockNormGrads(NamedTuple):
    dx: torch.Tensor
    dh: Optional[torch.Tensor]
    dpost_weight: Optional[torch.Tensor]
    dpost_bias: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dpre_weight: Optional[torch.Tensor]
    dpre_bias: Optional[torch.Tensor]


def block_norm(h: Optional[torch.Tensor], x: torch.Tensor, kind: str = "layer", post_norm: bool = False,
               post_weight: Optional[torch.Tensor] = None, post_bias: Optional[torch.Tensor] = None,
               gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0, pre_norm: bool = True,
               pre_weight: Optional[torch.Tensor] = None, pre_bias: Optional[torch.Tensor] = None,
               weight_offset: float = 0.0, eps: float = 1e-6, out: Optional[BlockNorm] = None,
               stream=None) -> BlockNorm:
    """The end of one block and the norm of the next in one pass over the rows:
    n = norm(h) * (post_weight + weight_offset) + post_bias (n = h without post_norm),
    x_out = residual_scale * x + gate * n, y = norm(x_out) * (pre_weight + weight_offset) + pre_bias.
    kind "layer" or "rms". h, x: rows x cols, both bf16 or fp32, any row stride; h None: no block output
    (the first norm; x_out is None then if residual_scale is 1). gate: cols, or groups x cols for
    consecutive groups of rows. stats (rows x 4 fp32) is what block_norm_backward needs."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return block_norm(h, x, kind, post_norm, post_weight, post_bias, gate, residual_scale, pre_norm,
                              pre_weight, pre_bias, weight_offset, eps, out)
    if _fast is not None and out is None:
        r = _fast.block_norm(h, x, NORM_KINDS.get(kind, 0), post_norm, post_weight, post_bias, gate, residual_scale,
                             pre_norm, pre_weight, pre_bias, weight_offset, eps)
        if r is not None:
            return BlockNorm(*_taken(r, "bsq_block_norm"))
    xs = _matrix(x, "x")
    rows, cols = x.shape
    hs = _matrix(h, "h", x.dtype, x.shape) if h is not None else 0
    assert h is not None or not (post_norm or gate is not None), "a post norm or a gate needs h"
    assert post_norm or (post_weight is None and post_bias is None), "post_weight / post_bias need post_norm"
    assert pre_norm or (pre_weight is None and pre_bias is None), "pre_weight / pre_bias need pre_norm"
    flags, groups = _params(cols, gate, (("post_weight", post_weight), ("post_bias", post_bias),
                                         ("pre_weight", pre_weight), ("pre_bias", pre_bias)))
    _on_current_device(h, x, post_weight, post_bias, gate, pre_weight, pre_bias, *(out or ()))
    if x.dtype is _F32:
        flags |= FLAG_SRC_F32
    if post_norm:
        flags |= FLAG_POST_NORM
    if out is not None:
        x_out, y, stats = out
        for t in (x_out, y):
            assert t is None or (t.shape == x.shape and t.dtype == x.dtype and t.is_cuda and t.is_contiguous()), \
                "out tensors must be contiguous CUDA tensors like x"
        assert pre_norm == (y is not None), "out.y goes with pre_norm"
        assert stats is None or (stats.shape == (rows, 4) and stats.dtype == torch.float32 and stats.is_cuda and
                                 stats.is_contiguous()), "out.stats must be rows x 4 float32"
    else:
        dt, dev = x.dtype, x.device
        x_out = torch.empty((rows, cols), dtype=dt, device=dev) \
            if h is not None or residual_scale != 1.0 or not pre_norm else None
        y = torch.empty((rows, cols), dtype=dt, device=dev) if pre_norm else None
        stats = torch.empty((rows, 4), dtype=_F32, device=dev)
    a = _NORM_ARGS.pack(NORM_KINDS[kind], flags, rows, cols, groups, eps, residual_scale, weight_offset, _addr(h),
                        x.data_ptr(), hs, xs, _addr(post_weight), _addr(post_bias), _addr(gate), _addr(pre_weight),
                        _addr(pre_bias), _addr(x_out), _addr(y), _addr(stats))
    rc = _lib.bsq_block_norm(a, _handle(x))
    if rc != OK:
        raise BsqError(rc, "bsq_block_norm")
    return BlockNorm(x_out, y, stats)


def block_norm_backward(dx_out: Optional[torch.Tensor], dy: Optional[torch.Tensor], x_out: Optional[torch.Tensor],
                        h: Optional[torch.Tensor], stats: torch.Tensor, kind: str = "layer", post_norm: bool = False,
                        post_weight: Optional[torch.Tensor] = None, post_bias: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                        pre_weight: Optional[torch.Tensor] = None, pre_bias: Optional[torch.Tensor] = None,
                        weight_offset: float = 0.0, param_grads: bool = True, stream=None) -> BlockNormGrads:
    """Gradients of block_norm from those of x_out and y (either may be None: zero). x_out (the
    forward's; x itself where the forward had neither h nor a scale) and stats are what the forward
    returned; the parameters are the forward's. dx, dh have the input's dtype, every parameter's
    gradient is fp32; None stands for the gradient of what was not given."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return block_norm_backward(dx_out, dy, x_out, h, stats, kind, post_norm, post_weight, post_bias, gate,
                                       residual_scale, pre_weight, pre_bias, weight_offset, param_grads)
    if _fast is not None:
        r = _fast.block_norm_backward(dx_out, dy, x_out, h, stats, NORM_KINDS.get(kind, 0), post_norm, post_weight,
                                      post_bias, gate, residual_scale, pre_weight, pre_bias, weight_offset, param_grads)
        if r is not None:
            return BlockNormGrads(*_taken(r, "bsq_block_norm_backward"))
    g = dy if dy is not None else dx_out
    assert g is not None, "dx_out or dy must be given"
    _matrix(g, "dy" if dy is not None else "dx_out")
    rows, cols = g.shape
    dys = _matrix(dy, "dy") if dy is not None else 0
    dxs = _matrix(dx_out, "dx_out", g.dtype, g.shape) if dx_out is not None else 0
    assert dy is None or x_out is not None, "dy needs x_out"
    xs = _matrix(x_out, "x_out", g.dtype, g.shape) if x_out is not None else 0
    hs = _matrix(h, "h", g.dtype, g.shape) if h is not None else 0
    assert h is not None or not (post_norm or gate is not None), "a post norm or a gate needs h"
    assert post_norm or (post_weight is None and post_bias is None), "post_weight / post_bias need post_norm"
    assert stats.shape == (rows, 4) and stats.dtype == torch.float32 and stats.is_cuda and stats.is_contiguous(), \
        "stats must be rows x 4 float32, as block_norm returns it"
    flags, groups = _params(cols, gate, (("post_weight", post_weight), ("post_bias", post_bias),
                                         ("pre_weight", pre_weight), ("pre_bias", pre_bias)))
    _on_current_device(dx_out, dy, x_out, h, stats, post_weight, post_bias, gate, pre_weight, pre_bias)
    if g.dtype is _F32:
        flags |= FLAG_SRC_F32
    if post_norm:
        flags |= FLAG_POST_NORM
    dt, dev = g.dtype, g.device
    dx = torch.empty((rows, cols), dtype=dt, device=dev)
    dh = torch.empty((rows, cols), dtype=dt, device=dev) if h is not None else None
    dp = [None] * 5
    ws, ws_bytes = None, 0
    if param_grads:
        n = 0
        for i, p in enumerate((post_weight, post_bias, gate, pre_weight if dy is not None else None,
                               pre_bias if dy is not None else None)):
            if p is not None:
                dp[i] = torch.empty(p.shape, dtype=_F32, device=dev)
                n += 1
        if n and rows > 0:
            ws_bytes = _lib.bsq_block_norm_backward_workspace(flags, rows, cols, groups)
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    a = _NORM_GRAD_ARGS.pack(NORM_KINDS[kind], flags, rows, cols, groups, residual_scale, weight_offset, _addr(dx_out),
                             _addr(dy), _addr(x_out), _addr(h), dxs, dys, xs, hs, stats.data_ptr(), _addr(post_weight),
                             _addr(post_bias), _addr(gate), _addr(pre_weight), _addr(pre_bias), dx.data_ptr(),
                             _addr(dh), _addr(dp[0]), _addr(dp[1]), _addr(dp[2]), _addr(dp[3]), _addr(dp[4]),
                             _addr(ws), ws_bytes)
    rc = _lib.bsq_block_norm_backward(a, _handle(g))
    if rc != OK:
        raise BsqError(rc, "bsq_block_norm_backward")
    return BlockNormGrads(dx, dh, *dp)


class ExpertSort(NamedTuple):
    counts: torch.Tensor
    offsets: torch.Tensor
    position: torch.Tensor
    slot: torch.Tensor


def _whole(x: torch.Tensor, what: str, dtype=torch.int32):
    if x.dtype is not dtype:
        raise TypeError("%s must be %s" % (what, dtype))
    assert x.is_cuda and x.is_contiguous(), "%s must be a contiguous CUDA tensor" % what


def expert_sort(ids: torch.Tensor, experts: int, align: int = 1, stream=None) -> ExpertSort:
    """Rows sorted by expert for a router's choices ids (tokens x topk, int32 or int64; ids outside
    [0, experts) are dropped): counts (experts), offsets (experts + 1; each expert's first row, a
    multiple of align), position (tokens x topk: the row of each choice, -1 if dropped) and slot
    (one for each row of the capacity: token * topk + j, -1 for a row of none), all int32. The
    capacity holds any choice of ids, so nothing is read back to the host."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return expert_sort(ids, experts, align)
    if _fast is not None:
        r = _fast.expert_sort(ids, experts, align)
        if r is not None:
            return ExpertSort(*_taken(r, "bsq_expert_sort"))
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be int32 or int64")
    assert ids.is_cuda and ids.is_contiguous() and ids.dim() == 2, "ids must be a contiguous 2-D CUDA tensor"
    _on_current_device(ids)
    tokens, topk = ids.shape
    slots, dev = tokens * topk, ids.device
    if topk < 1 or experts < 1 or align < 1:
        raise BsqError(ERR_ARG, "bsq_expert_sort")
    capacity = _lib.bsq_expert_capacity(slots, experts, align)
    if max(slots, align, capacity) >= 1 << 31 or experts > MAX_EXPERTS:  # before anything of such a size is allocated
        raise BsqError(ERR_SHAPE, "bsq_expert_sort")
    counts = torch.empty(experts, dtype=_I32, device=dev)
    offsets = torch.empty(experts + 1, dtype=_I32, device=dev)
    position = torch.empty((tokens, topk), dtype=_I32, device=dev)
    slot = torch.empty(capacity, dtype=_I32, device=dev)
    ws_bytes = _lib.bsq_expert_sort_workspace(slots, experts)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    rc = _lib.bsq_expert_sort(FLAG_IDS_I64 if ids.dtype is _I64 else 0, ids.data_ptr(), tokens, topk, experts, align,
                              capacity, counts.data_ptr(), offsets.data_ptr(), position.data_ptr(), slot.data_ptr(),
                              _addr(ws), ws_bytes, _handle(ids))
    if rc != OK:
        raise BsqError(rc, "bsq_expert_sort")
    return ExpertSort(counts, offsets, position, slot)


def expert_gather(x: torch.Tensor, position: torch.Tensor, slot: torch.Tensor, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """rows[r] = x[slot[r] // topk], zeros where slot[r] is -1: x (tokens x cols, bf16 or fp32) sorted by
    expert; position and slot are expert_sort's."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return expert_gather(x, position, slot, out)
    if _fast is not None and out is None:
        r = _fast.expert_gather(x, position, slot)
        if r is not None:
            return _taken(r, "bsq_expert_gather")
    xs = _matrix(x, "x")
    _whole(position, "position")
    _whole(slot, "slot")
    tokens, cols = x.shape
    assert position.dim() == 2 and position.shape[0] == tokens, "position must be tokens x topk"
    _on_current_device(x, position, slot, out)
    if out is None:
        out = torch.empty((slot.shape[0], cols), dtype=x.dtype, device=x.device)
    else:
        assert out.shape == (slot.shape[0], cols) and out.dtype == x.dtype and out.is_contiguous() and out.is_cuda
    rc = _lib.bsq_expert_gather(FLAG_SRC_F32 if x.dtype is _F32 else 0, x.data_ptr(), xs, position.data_ptr(),
                                slot.data_ptr(), tokens, position.shape[1], cols, slot.shape[0], out.data_ptr(), _handle(x))
    if rc != OK:
        raise BsqError(rc, "bsq_expert_gather")
    return out


def expert_combine(y: torch.Tensor, position: torch.Tensor, weights: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = sum over j of weights[t, j] * y[position[t, j]] (fp32 sums; dropped choices add nothing):
    the experts' rows back in token order. weights: tokens x topk fp32, None: 1."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return expert_combine(y, position, weights, out)
    if _fast is not None and out is None:
        r = _fast.expert_combine(y, position, weights)
        if r is not None:
            return _taken(r, "bsq_expert_combine")
    ys = _matrix(y, "y")
    _whole(position, "position")
    assert position.dim() == 2, "position must be tokens x topk"
    tokens, topk = position.shape
    if weights is not None:
        _whole(weights, "weights", torch.float32)
        assert weights.shape == position.shape, "weights must be tokens x topk"
    capacity, cols = y.shape
    _on_current_device(y, position, weights, out)
    if out is None:
        out = torch.empty((tokens, cols), dtype=y.dtype, device=y.device)
    else:
        assert out.shape == (tokens, cols) and out.dtype == y.dtype and out.is_contiguous() and out.is_cuda
    rc = _lib.bsq_expert_combine(FLAG_SRC_F32 if y.dtype is _F32 else 0, y.data_ptr(), ys, position.data_ptr(),
                                 _addr(weights), tokens, topk, cols, capacity, out.data_ptr(), _handle(y))
    if rc != OK:
        raise BsqError(rc, "bsq_expert_combine")
    return out


def expert_gather_backward(drows: torch.Tensor, position: torch.Tensor, out: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """Gradient of expert_gather: dx[t] = sum over j of drows[position[t, j]]."""
    return expert_combine(drows, position, None, out, stream)


def expert_combine_backward(dout: torch.Tensor, y: torch.Tensor, position: torch.Tensor, slot: torch.Tensor,
                            weights: torch.Tensor, stream=None):
    """Gradients of expert_combine: (dy, dweights), dy like y (zeros in rows of no slot), dweights
    tokens x topk fp32 (0 for dropped choices)."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return expert_combine_backward(dout, y, position, slot, weights)
    if _fast is not None:
        r = _fast.expert_combine_backward(dout, y, position, slot, weights)
        if r is not None:
            return _taken(r, "bsq_expert_combine_backward")
    ys = _matrix(y, "y")
    capacity, cols = y.shape
    _whole(position, "position")
    _whole(slot, "slot")
    _whole(weights, "weights", torch.float32)
    assert position.dim() == 2 and weights.shape == position.shape, "position and weights must be tokens x topk"
    assert slot.shape == (capacity,), "slot must have one value for each row of y"
    tokens, topk = position.shape
    ds = _matrix(dout, "dout", y.dtype, (tokens, cols))
    _on_current_device(dout, y, position, slot, weights)
    dy = torch.empty((capacity, cols), dtype=y.dtype, device=y.device)
    dweights = torch.empty((tokens, topk), dtype=torch.float32, device=y.device)
    rc = _lib.bsq_expert_combine_backward(FLAG_SRC_F32 if y.dtype is _F32 else 0, dout.data_ptr(), ds, y.data_ptr(), ys,
                                          position.data_ptr(), slot.data_ptr(), weights.data_ptr(), tokens, topk, cols,
                                          capacity, dy.data_ptr(), dweights.data_ptr(), _handle(y))
    if rc != OK:
        raise BsqError(rc, "bsq_expert_combine_backward")
    return dy, dweights


def _norm_kind(norm_type: float) -> int:
    if norm_type == 2:
        return GRAD_NORM_L2
    if norm_type == float("inf"):
        return GRAD_NORM_MAX
    raise ValueError("norm_type must be 2 or infinity")


def _grad_array(tensors, outs) -> array.array:
    """The bsq_grad_item array of the gradients as 64-bit words: src, dst, elems, f32. Attributes are
    collected by map over whole lists: hundreds of small tensors cost 0.5 us each, not 1.5."""
    tt = torch.Tensor
    f32 = [t.dtype is _F32 for t in tensors]
    if not all(f32) and any([not f and t.dtype is not _BF16 for f, t in zip(f32, tensors)]):
        raise TypeError("gradients must be bfloat16 or float32")
    elems = array.array("q", map(tt.numel, tensors))
    devices = set(map(tt.get_device, tensors))
    assert min(devices, default=0) >= 0 and all(map(tt.is_contiguous, tensors)), \
        "gradients must be contiguous CUDA tensors"
    words = array.array("q", bytes(32 * len(tensors)))
    words[0::4] = words[1::4] = array.array("q", map(tt.data_ptr, tensors))
    words[2::4] = elems
    words[3::4] = array.array("q", f32)
    if outs is not None:
        assert len(outs) == len(tensors), "outs must have one tensor for each gradient"
        assert min(map(tt.get_device, outs), default=0) >= 0 and all(map(tt.is_contiguous, outs)) and \
            array.array("q", map(tt.numel, outs)) == elems and f32 == [o.dtype is _F32 for o in outs] and \
            (all(f32) or not any([not f and o.dtype is not _BF16 for f, o in zip(f32, outs)])), \
            "outs must be contiguous CUDA tensors like the gradients"
        words[1::4] = array.array("q", map(tt.data_ptr, outs))
        devices.update(map(tt.get_device, outs))
    assert not devices or devices == {torch.cuda.current_device()}, "all tensors must be on the current device"
    return words


def _grad_call(tensors, outs, norm_type, clip):
    tensors, outs = list(tensors), None if outs is None else list(outs)
    if _fast is not None:
        r = _fast.grad_norm(tensors, outs, _norm_kind(norm_type), None if clip is None else clip[0],
                            0.0 if clip is None else clip[1])
        if r is not None:
            return _taken(r, "bsq_grad_norm" if clip is None else "bsq_clip_grad_norm")
    words = _grad_array(tensors, outs)
    dev = tensors[0].device if tensors else torch.device("cuda", torch.cuda.current_device())
    n = _lib.bsq_clip_grad_norm_workspace(len(tensors))
    norm = torch.empty((), dtype=_F32, device=dev)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    items = ctypes.cast(words.buffer_info()[0], ctypes.POINTER(GradItem))
    kind, handle = _norm_kind(norm_type), _handle(norm)
    if clip is None:
        rc = _lib.bsq_grad_norm(len(tensors), items, kind, norm.data_ptr(), ws.data_ptr(), n, handle)
    else:
        rc = _lib.bsq_clip_grad_norm(len(tensors), items, kind, clip[0], clip[1], norm.data_ptr(), ws.data_ptr(), n,
                                     handle)
    if rc != OK:
        raise BsqError(rc, "bsq_grad_norm" if clip is None else "bsq_clip_grad_norm")
    return norm


def grad_norm(tensors, norm_type: float = 2.0, stream=None) -> torch.Tensor:
    """The norm (2 or infinity) of all gradients taken as one vector: a one-element fp32 tensor on
    the device. tensors: contiguous bf16 / fp32 CUDA tensors, mixed at will."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return grad_norm(tensors, norm_type)
    return _grad_call(tensors, None, norm_type, None)


def clip_grad_norm(tensors, max_norm: float, norm_type: float = 2.0, eps: float = 1e-6, outs=None,
                   stream=None) -> torch.Tensor:
    """Scales the gradients by max_norm / (norm + eps), where that is below 1, in place or into `outs`, and returns
    their norm before that (a one-element fp32 tensor; nothing is read back to the host). A NaN
    norm makes every gradient NaN."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return clip_grad_norm(tensors, max_norm, norm_type, eps, outs)
    return _grad_call(tensors, outs, norm_type, (max_norm, eps))


def device_status(stream=None) -> int:
    return bsq_get_device_status(stream)
