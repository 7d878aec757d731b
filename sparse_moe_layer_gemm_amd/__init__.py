"""Python binding of libmoe.so, the gfx950 routed-MoE layer (see include/moe.h).

Argument marshalling only: every step of the layer runs in the HIP kernels of
libmoe.so. Tensors are PyTorch-ROCm device tensors (device memory and streams
are all torch provides); pointers, sizes and the current HIP stream are passed
through ctypes under the same function names as the C ABI. There is no
fallback: if the library is missing, importing this package raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch  # loads the HIP runtime that libmoe.so then shares

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_F32, MOE_BF16, MOE_FP8_E4M3, MOE_FP4_E2M1 = 0, 1, 2, 3
MOE_QMODE_W, MOE_QMODE_F8 = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
DTYPE_NAMES = {"f32": MOE_F32, "bf16": MOE_BF16, "fp8": MOE_FP8_E4M3, "fp4": MOE_FP4_E2M1}
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARGUMENT", 2: "MOE_ERR_UNSUPPORTED",
          3: "MOE_ERR_WORKSPACE_TOO_SMALL", 4: "MOE_ERR_LAUNCH"}

ENTRY_POINTS = ("moe_status_string", "moe_route_workspace_size", "moe_route",
                "moe_permute_workspace_size", "moe_permute", "moe_experts_workspace_size",
                "moe_experts", "moe_experts_rows16", "moe_finalize", "moe_finalize_rows16",
                "moe_finalize_norm", "moe_finalize_norm_rows16", "moe_forward_workspace_size",
                "moe_forward", "moe_forward_norm", "moe_forward_noalloc",
                "moe_hbm_read", "moe_grouped_gemm", "moe_grouped_wgrad", "moe_swiglu",
                "moe_swiglu_backward", "moe_finalize_backward", "moe_mxfp4_scale_stride",
                "moe_mxfp4_quantize", "moe_mxfp4_dequantize", "moe_mxfp4_grouped_gemm", "moe_select",
                "moe_select_backward", "moe_w4_quantize", "moe_w4_dequantize", "moe_w4_grouped_gemm")


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


class CExpertWeights(ctypes.Structure):
    """struct moe_expert_weights"""
    _fields_ = [("dtype", ctypes.c_int32), ("qmode", ctypes.c_int32),
                ("gate_up", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("gate_up_scale", ctypes.c_void_p), ("down_scale", ctypes.c_void_p),
                ("gate_up_gscale", ctypes.c_void_p), ("down_gscale", ctypes.c_void_p)]


_lib = None
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


def load_library(path: str = LIB_PATH):
    """Load libmoe.so (built by sparse_moe_layer_gemm_amd/build.py)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python sparse_moe_layer_gemm_amd/build.py`")
    lib = ctypes.CDLL(path)
    sig = {
        "moe_status_string": (ctypes.c_char_p, [_i32]),
        "moe_route_workspace_size": (_sz, [_i64, _i32, _i32]),
        "moe_route": (_i32, [_vp, _i32, _i64, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                             _vp, _sz, _vp]),
        "moe_permute_workspace_size": (_sz, [_i64, _i32, _i32]),
        "moe_permute": (_i32, [_vp, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
        "moe_experts_workspace_size": (_sz, [_i64, _i32, _i32, _i32, _i32, ctypes.POINTER(CExpertWeights)]),
        "moe_experts": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _i32, _vp, _vp,
                               ctypes.POINTER(CExpertWeights), _vp, _vp, _sz, _vp]),
        "moe_finalize": (_i32, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp]),
        "moe_experts_rows16": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _i32, _vp, _vp,
                                      ctypes.POINTER(CExpertWeights), _vp, _vp, _vp, _sz, _vp]),
        "moe_finalize_rows16": (_i32, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp]),
        "moe_finalize_norm": (_i32, [_vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp, _vp, ctypes.c_float,
                                     _vp, _vp, _vp]),
        "moe_finalize_norm_rows16": (_i32, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp, _vp,
                                            ctypes.c_float, _vp, _vp, _vp]),
        "moe_forward_norm": (_i32, [_vp, _i64, _i32, _i32, _i32, _i32, _vp, _vp,
                                    ctypes.POINTER(CExpertWeights), _vp, _vp, _vp, ctypes.c_float,
                                    _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
        "moe_forward_workspace_size": (_sz, [_i64, _i32, _i32, _i32, _i32, ctypes.POINTER(CExpertWeights)]),
        "moe_forward": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _i32, _vp, _vp,
                               ctypes.POINTER(CExpertWeights), _i32, _vp, _vp, _i32, _vp, _vp, _vp,
                               _vp, _sz, _vp]),
        "moe_forward_noalloc": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _i32, _vp, _vp,
                                       ctypes.POINTER(CExpertWeights), _i32, _vp, _vp, _i32, _vp,
                                       _vp, _vp, _vp]),
        "moe_hbm_read": (_i32, [_vp, _sz, _vp, _vp]),
        "moe_grouped_gemm": (_i32, [_vp, _i32, _i64, _vp, _i32, _vp, _i32, _i64, _i32, _i32, _i32,
                                    _vp, _i32, _vp, _vp]),
        "moe_grouped_wgrad": (_i32, [_vp, _i32, _i64, _vp, _i32, _vp, _i64, _i32, _i32, _i32, _vp,
                                     _i32, _i32, _vp, _vp]),
        "moe_swiglu": (_i32, [_vp, _i32, _i64, _i32, _vp, _vp]),
        "moe_swiglu_backward": (_i32, [_vp, _vp, _i32, _i64, _i32, _vp, _vp, _vp]),
        "moe_finalize_backward": (_i32, [_vp, _i32, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp,
                                         _vp]),
        "moe_mxfp4_scale_stride": (_i32, [_i32]),
        "moe_mxfp4_quantize": (_i32, [_vp, _i32, _i32, _i64, _i64, _i32, _vp, _vp, _vp]),
        "moe_mxfp4_dequantize": (_i32, [_vp, _vp, _i64, _i32, _i32, _vp, _vp]),
        "moe_mxfp4_grouped_gemm": (_i32, [_vp, _vp, _i64, _vp, _i32, _vp, _vp, _i64, _i32, _i32,
                                          _i32, _vp, _i32, _vp, _vp]),
        "moe_select": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _vp, _i32, _i32, _i32, _i32,
                              ctypes.c_float, _vp, _vp, _vp, _vp]),
        "moe_select_backward": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _i32, ctypes.c_float, _vp,
                                       _vp, _vp, _i32, _vp, _vp]),
        "moe_w4_quantize": (_i32, [_vp, _i32, _i32, _i64, _i64, _i32, _i32, _vp, _i32, _vp, _vp, _vp]),
        "moe_w4_dequantize": (_i32, [_vp, _i32, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp]),
        "moe_w4_grouped_gemm": (_i32, [_vp, _i64, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _i64, _i32,
                                       _i32, _i32, _vp, _i32, _vp, _vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    _lib = lib
    return lib


load_library()


# ---------------------------------------------------------------- marshalling helpers
def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise TypeError(f"unsupported tensor dtype {t.dtype}")


def _check(fn: str, status: int):
    if status != 0:
        raise MoEError(fn, status)


_I32_MAX = (1 << 31) - 1  # ctypes passes larger values on modulo 2^32, past the library's checks


def _too_wide(fn: str):
    raise ValueError(f"{fn}: every size but a number of rows must be below 2^31")


def _int32s(fn: str, *values):
    for v in values:
        if abs(v) > _I32_MAX:
            _too_wide(fn)


@dataclasses.dataclass
class ExpertWeights:
    """Device expert weights of one layer (layouts in include/moe.h)."""
    dtype: int
    gate_up: torch.Tensor
    down: torch.Tensor
    gate_up_scale: Optional[torch.Tensor] = None
    down_scale: Optional[torch.Tensor] = None
    gate_up_gscale: Optional[torch.Tensor] = None
    down_gscale: Optional[torch.Tensor] = None
    qmode: int = MOE_QMODE_W

    def c_struct(self) -> CExpertWeights:
        return CExpertWeights(self.dtype, self.qmode, _ptr(self.gate_up), _ptr(self.down),
                              _ptr(self.gate_up_scale), _ptr(self.down_scale),
                              _ptr(self.gate_up_gscale), _ptr(self.down_gscale))


# ---------------------------------------------------------------- the C ABI, same names
def moe_route_workspace_size(T: int, H: int, E: int) -> int:
    _int32s("moe_route_workspace_size", H, E)
    return _lib.moe_route_workspace_size(T, H, E)


def moe_route(x, w_router, bias, k: int, logits_dtype: int, logits, logits_f32, topk_ids, topk_w,
              workspace, stream=None):
    T, H = x.shape
    E = w_router.shape[1]
    _int32s("moe_route", H, E, k)
    _check("moe_route", _lib.moe_route(
        _ptr(x), _dt(x), T, H, _ptr(w_router), _ptr(bias), E, k, logits_dtype, _ptr(logits),
        _ptr(logits_f32), _ptr(topk_ids), _ptr(topk_w), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_permute_workspace_size(T: int, k: int, E: int) -> int:
    _int32s("moe_permute_workspace_size", k, E)
    return _lib.moe_permute_workspace_size(T, k, E)


def moe_permute(topk_ids, E: int, counts, offsets, sorted_pair, pair_pos, workspace=None,
                stream=None):
    T, k = topk_ids.shape
    _int32s("moe_permute", k, E)
    if workspace is None:
        need = moe_permute_workspace_size(T, k, E)
        workspace = globals()["workspace"](need, topk_ids.device) if need else None
    _check("moe_permute", _lib.moe_permute(
        _ptr(topk_ids), T, k, E, _ptr(counts), _ptr(offsets), _ptr(sorted_pair), _ptr(pair_pos),
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream)))


def moe_experts_workspace_size(T: int, H: int, I: int, E: int, k: int, w: ExpertWeights) -> int:
    _int32s("moe_experts_workspace_size", H, I, E, k)
    s = w.c_struct()
    return _lib.moe_experts_workspace_size(T, H, I, E, k, ctypes.byref(s))


def moe_experts(x, I: int, E: int, k: int, offsets, sorted_pair, w: ExpertWeights, y_sorted,
                workspace, stream=None):
    T, H = x.shape
    _int32s("moe_experts", H, I, E, k)
    s = w.c_struct()
    _check("moe_experts", _lib.moe_experts(
        _ptr(x), _dt(x), T, H, I, E, k, _ptr(offsets), _ptr(sorted_pair), ctypes.byref(s),
        _ptr(y_sorted), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def moe_experts_rows16(x, I: int, E: int, k: int, offsets, sorted_pair, w: ExpertWeights, y16,
                       y16_scale, workspace, stream=None):
    """y16 [T*k, H] int16/uint16 (fp16 bits), y16_scale [T*k, H/64] uint8."""
    T, H = x.shape
    _int32s("moe_experts_rows16", H, I, E, k)
    s = w.c_struct()
    _check("moe_experts_rows16", _lib.moe_experts_rows16(
        _ptr(x), _dt(x), T, H, I, E, k, _ptr(offsets), _ptr(sorted_pair), ctypes.byref(s),
        _ptr(y16), _ptr(y16_scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def moe_finalize_rows16(y16, y16_scale, pair_pos, topk_w, out, out_f32=None, stream=None):
    T, k = topk_w.shape
    H = y16.shape[1]
    _int32s("moe_finalize_rows16", k, H)
    _check("moe_finalize_rows16", _lib.moe_finalize_rows16(
        _ptr(y16), _ptr(y16_scale), _ptr(pair_pos), _ptr(topk_w), T, k, H, _dt(out), _ptr(out),
        _ptr(out_f32), _stream(stream)))


def moe_finalize(y_sorted, pair_pos, topk_w, out, out_f32=None, stream=None):
    T, k = topk_w.shape
    H = y_sorted.shape[1]
    _int32s("moe_finalize", k, H)
    _check("moe_finalize", _lib.moe_finalize(
        _ptr(y_sorted), _ptr(pair_pos), _ptr(topk_w), T, k, H, _dt(out), _ptr(out), _ptr(out_f32),
        _stream(stream)))


def moe_finalize_norm(y_sorted, pair_pos, topk_w, residual, gamma_post, gamma_next, eps: float,
                      residual_out, normed, stream=None):
    """residual, residual_out, normed: [T, H] bf16 (residual_out may be residual);
    gamma_post, gamma_next: [H] bf16."""
    T, k = topk_w.shape
    H = y_sorted.shape[1]
    for t in (residual, gamma_post, gamma_next, residual_out, normed):
        if t.dtype != torch.bfloat16:
            raise ValueError("moe_finalize_norm takes bf16 residual, norm weights and outputs")
    _int32s("moe_finalize_norm", k, H)
    _check("moe_finalize_norm", _lib.moe_finalize_norm(
        _ptr(y_sorted), _ptr(pair_pos), _ptr(topk_w), T, k, H, _ptr(residual), _ptr(gamma_post),
        _ptr(gamma_next), float(eps), _ptr(residual_out), _ptr(normed), _stream(stream)))


def moe_finalize_norm_rows16(y16, y16_scale, pair_pos, topk_w, residual, gamma_post, gamma_next,
                             eps: float, residual_out, normed, stream=None):
    """moe_finalize_norm over compact rows (y16 [T*k, H] fp16 bits, y16_scale [T*k, H/64])."""
    T, k = topk_w.shape
    H = y16.shape[1]
    for t in (residual, gamma_post, gamma_next, residual_out, normed):
        if t.dtype != torch.bfloat16:
            raise ValueError("moe_finalize_norm_rows16 takes bf16 residual, norm weights and outputs")
    _int32s("moe_finalize_norm_rows16", k, H)
    _check("moe_finalize_norm_rows16", _lib.moe_finalize_norm_rows16(
        _ptr(y16), _ptr(y16_scale), _ptr(pair_pos), _ptr(topk_w), T, k, H, _ptr(residual),
        _ptr(gamma_post), _ptr(gamma_next), float(eps), _ptr(residual_out), _ptr(normed),
        _stream(stream)))


def moe_forward_workspace_size(T: int, H: int, I: int, E: int, k: int, w: ExpertWeights) -> int:
    _int32s("moe_forward_workspace_size", H, I, E, k)
    s = w.c_struct()
    return _lib.moe_forward_workspace_size(T, H, I, E, k, ctypes.byref(s))


def moe_forward(x, w_router, bias, w: ExpertWeights, I: int, k: int, out, workspace,
                out_f32=None, logits_dtype: Optional[int] = None, logits=None, topk_ids=None,
                topk_w=None, stream=None):
    T, H = x.shape
    E = w_router.shape[1]
    if logits_dtype is None:
        logits_dtype = _dt(x)
    _int32s("moe_forward", H, I, E, k)
    s = w.c_struct()
    _check("moe_forward", _lib.moe_forward(
        _ptr(x), _dt(x), T, H, I, E, k, _ptr(w_router), _ptr(bias), ctypes.byref(s), _dt(out),
        _ptr(out), _ptr(out_f32), logits_dtype, _ptr(logits), _ptr(topk_ids), _ptr(topk_w),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_forward_norm(x, w_router, bias, w: ExpertWeights, I: int, k: int, residual, gamma_post,
                     gamma_next, eps: float, residual_out, normed, workspace, logits=None,
                     topk_ids=None, topk_w=None, stream=None):
    """The layer ending in the fused finalize + sandwich norms (bf16 x, residual and outputs)."""
    T, H = x.shape
    E = w_router.shape[1]
    for t in (x, residual, gamma_post, gamma_next, residual_out, normed):
        if t.dtype != torch.bfloat16:
            raise ValueError("moe_forward_norm takes bf16 x, residual, norm weights and outputs")
    _int32s("moe_forward_norm", H, I, E, k)
    s = w.c_struct()
    _check("moe_forward_norm", _lib.moe_forward_norm(
        _ptr(x), T, H, I, E, k, _ptr(w_router), _ptr(bias), ctypes.byref(s), _ptr(residual),
        _ptr(gamma_post), _ptr(gamma_next), float(eps), _ptr(residual_out), _ptr(normed),
        _ptr(logits), _ptr(topk_ids), _ptr(topk_w), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 64 << 20  # MOE_NOALLOC_SCRATCH_BYTES


def moe_forward_noalloc(x, w_router, bias, w: ExpertWeights, I: int, k: int, out, out_f32=None,
                        logits_dtype: Optional[int] = None, logits=None, topk_ids=None, topk_w=None,
                        stream=None):
    """moe_forward on the library's own scratch area (no workspace argument, no allocation)."""
    T, H = x.shape
    E = w_router.shape[1]
    if logits_dtype is None:
        logits_dtype = _dt(x)
    _int32s("moe_forward_noalloc", H, I, E, k)
    s = w.c_struct()
    _check("moe_forward_noalloc", _lib.moe_forward_noalloc(
        _ptr(x), _dt(x), T, H, I, E, k, _ptr(w_router), _ptr(bias), ctypes.byref(s), _dt(out),
        _ptr(out), _ptr(out_f32), logits_dtype, _ptr(logits), _ptr(topk_ids), _ptr(topk_w),
        _stream(stream)))


# ---------------------------------------------------------------- operators around the layer
# A small call is bound by its host side, so these check in line and touch each tensor once.
# current_stream() builds an object, 2.7 us a call; torch's private names do not, where it has them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", lambda: torch.cuda.current_device())
_FLOATS = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}


def _refuse(fn: str, what: str):
    raise ValueError(f"{fn}: {what}")


def _float(t: torch.Tensor) -> int:
    d = _FLOATS.get(t.dtype)
    return _dt(t) if d is None else d  # _dt raises


def _arrays(fn: str, tensors):
    """Addresses of tensors (None for None), all contiguous and on one GPU, and that GPU's index."""
    index, at = None, []
    for t in tensors:
        if t is None:
            at.append(None)
            continue
        d = t.get_device()
        if d != index:
            if d < 0:
                _refuse(fn, "takes device tensors")
            if index is not None:
                _refuse(fn, "tensors on different devices")
            index = d
        if not t.is_contiguous():
            _refuse(fn, "tensors must be contiguous")
        at.append(t.data_ptr())
    return index, at


def _run(fn: str, call, index: int, stream, *args):
    """One call of the C ABI on GPU `index`, on the given stream or that GPU's current one."""
    raw = _raw_stream(index) if stream is None else _stream(stream)
    if index == _current_device():
        status = call(*args, raw)
    else:
        with torch.cuda.device(index):
            status = call(*args, raw)
    if status:
        raise MoEError(fn, status)


def _check_rows(fn, M, E, offsets, row_index, row_div):
    if offsets.dtype is not torch.int32 or offsets.shape != (E + 1,):
        _refuse(fn, "offsets must be int32 [E + 1]")
    if row_index is not None:
        if row_index.dtype is not torch.int32 or row_index.numel() != M:
            _refuse(fn, "row_index must be int32 [M]")
        if row_div < 1:
            _refuse(fn, "row_div must be positive")
        if row_div > _I32_MAX:
            _too_wide(fn)


def moe_grouped_gemm(a, w, offsets, out, row_index=None, row_div: int = 1, w_trans: bool = False,
                     stream=None):
    """out[r] = a[row_index[r] // row_div] @ w[e] for the rows r of each expert e (offsets, as
    moe_permute writes them). a [rows, K], w [E, K, N] (w_trans: [E, N, K]), out [M, N]. The
    input gradient is the same call on the output gradient with w_trans flipped."""
    fn = "moe_grouped_gemm"
    sa, sw, so = a.shape, w.shape, out.shape
    if len(sa) != 2 or len(sw) != 3 or len(so) != 2:
        _refuse(fn, "a and out are matrices, w [E, ., .]")
    (rows, K), (M, N), E = sa, so, sw[0]
    if sw != ((E, N, K) if w_trans else (E, K, N)):
        _refuse(fn, "shapes of a, w and out do not match")
    if w.dtype is not a.dtype:
        _refuse(fn, "a and w must have one dtype")
    if (K | N | E) > _I32_MAX:
        _too_wide(fn)
    _check_rows(fn, M, E, offsets, row_index, row_div)
    t_in, t_out = _float(a), _float(out)
    dev, (pa, pw, po, pout, pi) = _arrays(fn, (a, w, offsets, out, row_index))
    _run(fn, _lib.moe_grouped_gemm, dev, stream, pa, t_in, rows, pi, row_div, pw,
         1 if w_trans else 0, M, K, N, E, po, t_out, pout)


def moe_grouped_wgrad(a, d, offsets, dw, row_index=None, row_div: int = 1, accumulate: bool = False,
                      stream=None):
    """dw[e] = sum over expert e's rows r of a[row_index[r] // row_div]^T d[r] (accumulate: added
    to dw, fp32). a [rows, K], d [M, N], dw [E, K, N]."""
    fn = "moe_grouped_wgrad"
    sa, sd, sw = a.shape, d.shape, dw.shape
    if len(sa) != 2 or len(sd) != 2 or len(sw) != 3:
        _refuse(fn, "a and d are matrices, dw [E, K, N]")
    (rows, K), (M, N), E = sa, sd, sw[0]
    if sw != (E, K, N):
        _refuse(fn, "shapes of a, d and dw do not match")
    if a.dtype is not d.dtype:
        _refuse(fn, "a and d must have one dtype")
    if (K | N | E) > _I32_MAX:
        _too_wide(fn)
    _check_rows(fn, M, E, offsets, row_index, row_div)
    t_in, t_out = _float(a), _float(dw)
    dev, (pa, pd, po, pw, pi) = _arrays(fn, (a, d, offsets, dw, row_index))
    _run(fn, _lib.moe_grouped_wgrad, dev, stream, pa, t_in, rows, pi, row_div, pd, M, K, N, E,
         po, t_out, 1 if accumulate else 0, pw)


def moe_swiglu(a, h, stream=None):
    """h = silu(a[:, :I]) * a[:, I:]; a [M, 2I], h [M, I], bf16 or fp32."""
    fn = "moe_swiglu"
    sh = h.shape
    if len(sh) != 2 or a.shape != (sh[0], 2 * sh[1]):
        _refuse(fn, "a must be [M, 2I] and h [M, I]")
    if a.dtype is not h.dtype:
        _refuse(fn, "a and h must have one dtype")
    if sh[1] > _I32_MAX:
        _too_wide(fn)
    t_in = _float(a)
    dev, (pa, ph) = _arrays(fn, (a, h))
    _run(fn, _lib.moe_swiglu, dev, stream, pa, t_in, sh[0], sh[1], ph)


def moe_swiglu_backward(a, dh, da, h=None, stream=None):
    """da [M, 2I] = gradient of moe_swiglu at a for dh [M, I]; h [M, I], if given, is formed again.
    da may be a and h may be dh."""
    fn = "moe_swiglu_backward"
    sh, t = dh.shape, a.dtype
    if len(sh) != 2 or a.shape != (sh[0], 2 * sh[1]):
        _refuse(fn, "a must be [M, 2I] and dh [M, I]")
    if da.shape != a.shape or (h is not None and h.shape != sh):
        _refuse(fn, "da is shaped as a, h as dh")
    if dh.dtype is not t or da.dtype is not t or (h is not None and h.dtype is not t):
        _refuse(fn, "all tensors must have one dtype")
    if sh[1] > _I32_MAX:
        _too_wide(fn)
    t_in = _float(a)
    dev, (pa, pdh, pda, ph) = _arrays(fn, (a, dh, da, h))
    _run(fn, _lib.moe_swiglu_backward, dev, stream, pa, pdh, t_in, sh[0], sh[1], pda, ph)


def moe_finalize_backward(dout, y_sorted, pair_pos, topk_w, dy_sorted, dtopk_w, stream=None):
    """Gradients of moe_finalize: dy_sorted[pair_pos] = topk_w * dout, dtopk_w = <dout, y_sorted[pair_pos]>
    (either output may be None; y_sorted may be None without dtopk_w)."""
    fn = "moe_finalize_backward"
    sd, sw = dout.shape, topk_w.shape
    if len(sd) != 2 or len(sw) != 2 or sw[0] != sd[0] or topk_w.dtype is not torch.float32:
        _refuse(fn, "dout must be [T, H] and topk_w fp32 [T, k]")
    (T, H), k = sd, sw[1]
    if (H | k) > _I32_MAX:
        _too_wide(fn)
    if pair_pos.dtype is not torch.int32 or pair_pos.numel() != T * k:
        _refuse(fn, "pair_pos must be int32 [T*k]")
    if y_sorted is not None and (y_sorted.dtype is not torch.float32 or y_sorted.shape != (T * k, H)):
        _refuse(fn, "y_sorted must be fp32 [T*k, H]")
    if dy_sorted is not None and dy_sorted.shape != (T * k, H):
        _refuse(fn, "dy_sorted must be [T*k, H]")
    if dtopk_w is not None and (dtopk_w.dtype is not torch.float32 or dtopk_w.shape != sw):
        _refuse(fn, "dtopk_w must be fp32 [T, k]")
    t_in, t_out = _float(dout), MOE_F32 if dy_sorted is None else _float(dy_sorted)
    dev, (pd, py, pp, pw, pdy, pdw) = _arrays(fn, (dout, y_sorted, pair_pos, topk_w, dy_sorted, dtopk_w))
    _run(fn, _lib.moe_finalize_backward, dev, stream, pd, t_in, py, pp, pw, T, k, H,
         t_out, pdy, pdw)


def moe_mxfp4_scale_stride(K: int) -> int:
    """Scale bytes per row of K MXFP4 values: K / 32 rounded up to a multiple of 4."""
    _int32s("moe_mxfp4_scale_stride", K)
    return _lib.moe_mxfp4_scale_stride(K)


def _check_mx(fn, codes, scales, rows, K):
    if K % 32 or codes.dtype is not torch.uint8 or codes.shape != (*rows, K // 2):
        _refuse(fn, "codes must be uint8 [rows, K/2], K a multiple of 32")
    if scales.dtype is not torch.uint8 or scales.shape != (*rows, (K // 32 + 3) // 4 * 4):
        _refuse(fn, "scales must be uint8 [rows, moe_mxfp4_scale_stride(K)]")


def moe_mxfp4_quantize(x, codes, scales, trans: bool = False, stream=None):
    """MXFP4 of x [..., K] along its last dimension: codes [..., K/2], scales [..., S]. With trans,
    x [B, K, C] (or [K, C]) along its middle dimension: codes [B, C, K/2], scales [B, C, S]."""
    fn = "moe_mxfp4_quantize"
    sx = x.shape
    if len(sx) == 2:
        B, (R, C) = 1, sx
        _check_mx(fn, codes, scales, (C,) if trans else (R,), R if trans else C)
    elif len(sx) == 3:
        B, R, C = sx
        _check_mx(fn, codes, scales, (B, C) if trans else (B, R), R if trans else C)
    else:
        _refuse(fn, "x must have two or three dimensions")
    if C > _I32_MAX:
        _too_wide(fn)
    t_in = _float(x)
    dev, (px, pc, ps) = _arrays(fn, (x, codes, scales))
    _run(fn, _lib.moe_mxfp4_quantize, dev, stream, px, t_in, 1 if trans else 0, B, R, C, pc, ps)


def moe_mxfp4_dequantize(codes, scales, out, stream=None):
    """out [..., K] (bf16 or fp32) = the values of codes [..., K/2] under scales [..., S]."""
    fn = "moe_mxfp4_dequantize"
    so = out.shape
    if not so:
        _refuse(fn, "out must be [..., K]")
    K = so[-1]
    _check_mx(fn, codes, scales, so[:-1], K)
    if K > _I32_MAX:
        _too_wide(fn)
    t_out = _float(out)
    dev, (pc, ps, po) = _arrays(fn, (codes, scales, out))
    _run(fn, _lib.moe_mxfp4_dequantize, dev, stream, pc, ps, out.numel() // max(K, 1), K, t_out, po)


def moe_mxfp4_grouped_gemm(a_codes, a_scales, w_codes, w_scales, offsets, out, row_index=None,
                           row_div: int = 1, stream=None):
    """moe_grouped_gemm of MXFP4 rows a ([rows, K/2] codes, [rows, S] scales) and weights
    ([E, N, K/2], [E, N, S]); out [M, N] bf16 or fp32."""
    fn = "moe_mxfp4_grouped_gemm"
    sa, sw, so = a_codes.shape, w_codes.shape, out.shape
    if len(sa) != 2 or len(sw) != 3 or len(so) != 2:
        _refuse(fn, "a_codes and out are matrices, w_codes [E, N, K/2]")
    (rows, half), (M, N), E = sa, so, sw[0]
    if (2 * half | N | E) > _I32_MAX:
        _too_wide(fn)
    _check_mx(fn, a_codes, a_scales, (rows,), 2 * half)
    _check_mx(fn, w_codes, w_scales, (E, N), 2 * half)
    _check_rows(fn, M, E, offsets, row_index, row_div)
    t_out = _float(out)
    dev, (pa, psa, pw, psw, po, pout, pi) = _arrays(
        fn, (a_codes, a_scales, w_codes, w_scales, offsets, out, row_index))
    _run(fn, _lib.moe_mxfp4_grouped_gemm, dev, stream, pa, psa, rows, pi, row_div, pw, psw, M,
         2 * half, N, E, po, t_out, pout)


def _check_select(fn, logits, topk_ids, per_slot, score):
    """(T, E, k, score) of a routing call; per_slot: the fp32 [T, k] beside the ids."""
    sl, si = logits.shape, topk_ids.shape
    if len(sl) != 2 or len(si) != 2 or si[0] != sl[0]:
        _refuse(fn, "logits must be [T, E] and topk_ids [T, k]")
    if topk_ids.dtype is not torch.int32 or per_slot.dtype is not torch.float32 or per_slot.shape != si:
        _refuse(fn, "topk_ids must be int32 and the weights (or their gradient) fp32, [T, k]")
    if (sl[1] | si[1]) > _I32_MAX:
        _too_wide(fn)
    kind = _SCORES.get(score)
    if kind is None:
        _refuse(fn, "score must be 'softmax' or 'sigmoid'")
    return sl[0], sl[1], si[1], kind


def moe_select(logits, topk_ids, topk_w, score="softmax", bias=None, groups: int = 1, group_k: int = 1,
               group_top: int = 1, renorm: bool = True, scale: float = 1.0, scores=None, stream=None):
    """The k experts of each token by scores of logits [T, E] (bf16 or fp32) and their weights:
    topk_ids int32 [T, k] (-1: no expert left), topk_w fp32 [T, k]. score: "softmax" or "sigmoid";
    bias: fp32 [E], added to the scores for the choice; groups: the experts come from the group_k of
    that many groups whose group_top (1 or 2) largest choices sum highest; renorm: weights divided
    by their sum; scores: fp32 [T, E], receives all scores."""
    fn = "moe_select"
    T, E, k, kind = _check_select(fn, logits, topk_ids, topk_w, score)
    if bias is not None and (bias.dtype is not torch.float32 or bias.shape != (E,)):
        _refuse(fn, "bias must be fp32 [E]")
    if scores is not None and (scores.dtype is not torch.float32 or scores.shape != (T, E)):
        _refuse(fn, "scores must be fp32 [T, E]")
    _int32s(fn, groups, group_k, group_top)
    t_in = _float(logits)
    dev, (pl, pi, pw, pb, ps) = _arrays(fn, (logits, topk_ids, topk_w, bias, scores))
    _run(fn, _lib.moe_select, dev, stream, pl, t_in, T, E, k, kind, pb, groups, group_k, group_top,
         1 if renorm else 0, scale, pi, pw, ps)


def moe_select_backward(logits, topk_ids, dtopk_w, dlogits, score="softmax", renorm: bool = True,
                        scale: float = 1.0, dscores=None, stream=None):
    """dlogits [T, E] (bf16 or fp32) of moe_select's weights for dtopk_w fp32 [T, k] and, if given,
    of its scores for dscores fp32 [T, E]; the choice (topk_ids) is held fixed."""
    fn = "moe_select_backward"
    T, E, k, kind = _check_select(fn, logits, topk_ids, dtopk_w, score)
    if dlogits.shape != (T, E):
        _refuse(fn, "dlogits must be [T, E]")
    if dscores is not None and (dscores.dtype is not torch.float32 or dscores.shape != (T, E)):
        _refuse(fn, "dscores must be fp32 [T, E]")
    t_in, t_out = _float(logits), _float(dlogits)
    dev, (pl, pi, pw, ps, pd) = _arrays(fn, (logits, topk_ids, dtopk_w, dscores, dlogits))
    _run(fn, _lib.moe_select_backward, dev, stream, pl, t_in, T, E, k, kind, 1 if renorm else 0,
         scale, pi, pw, ps, t_out, pd)


def _check_w4(fn, codes, scales, zeros, rows, K) -> int:
    """The group of codes [rows, K/2] and scales (and zeros) [rows, K/G]."""
    if codes.dtype is not torch.uint8 or K % 32 or codes.shape != (*rows, K // 2):
        _refuse(fn, "codes must be uint8 [rows, K/2], K a multiple of 32")
    ss = scales.shape
    if len(ss) != len(rows) + 1 or ss[:-1] != rows or ss[-1] < 1 or K % ss[-1]:
        _refuse(fn, "scales must be [rows, K/G]")
    if zeros is not None and (zeros.dtype is not torch.uint8 or zeros.shape != ss):
        _refuse(fn, "zeros must be uint8, shaped as scales")
    return K // ss[-1]


def moe_w4_quantize(x, codes, scales, zeros=None, trans: bool = False, stream=None):
    """4-bit codes of x [..., K] in groups along its last dimension: codes uint8 [..., K/2], scales (bf16 or
    fp32) [..., K/G], whose shape gives G (32, 64 or 128), and, if given, zero points uint8 [..., K/G]. With
    trans, x [B, K, C] (or [K, C]) along its middle dimension: codes [B, C, K/2] and so on."""
    fn = "moe_w4_quantize"
    sx = x.shape
    if len(sx) == 2:
        B, (R, C) = 1, sx
        rows, K = ((C,), R) if trans else ((R,), C)
    elif len(sx) == 3:
        B, R, C = sx
        rows, K = ((B, C), R) if trans else ((B, R), C)
    else:
        _refuse(fn, "x must have two or three dimensions")
    group = _check_w4(fn, codes, scales, zeros, rows, K)
    if (C | group) > _I32_MAX:
        _too_wide(fn)
    t_in, t_s = _float(x), _float(scales)
    dev, (px, pc, ps, pz) = _arrays(fn, (x, codes, scales, zeros))
    _run(fn, _lib.moe_w4_quantize, dev, stream, px, t_in, 1 if trans else 0, B, R, C, group, pc, t_s, ps, pz)


def moe_w4_dequantize(codes, scales, out, zeros=None, stream=None):
    """out [..., K] (bf16 or fp32) = (codes - zeros) * scales (zeros None: 8)."""
    fn = "moe_w4_dequantize"
    so = out.shape
    if not so:
        _refuse(fn, "out must be [..., K]")
    K = so[-1]
    group = _check_w4(fn, codes, scales, zeros, so[:-1], K)
    if K > _I32_MAX:
        _too_wide(fn)
    t_out, t_s = _float(out), _float(scales)
    dev, (pc, ps, pz, po) = _arrays(fn, (codes, scales, zeros, out))
    _run(fn, _lib.moe_w4_dequantize, dev, stream, pc, t_s, ps, pz, out.numel() // max(K, 1), K, group, t_out, po)


def moe_w4_grouped_gemm(a, w_codes, w_scales, offsets, out, zeros=None, row_index=None, row_div: int = 1,
                        stream=None):
    """moe_grouped_gemm of bf16 rows a [rows, K] and 4-bit weights: codes [E, N, K/2], scales [E, N, K/G]
    and, if given, zero points [E, N, K/G]; out [M, N] bf16 or fp32."""
    fn = "moe_w4_grouped_gemm"
    sa, sw, so = a.shape, w_codes.shape, out.shape
    if len(sa) != 2 or len(sw) != 3 or len(so) != 2:
        _refuse(fn, "a and out are matrices, w_codes [E, N, K/2]")
    if a.dtype is not torch.bfloat16:
        _refuse(fn, "a must be bf16")
    (rows, K), (M, N), E = sa, so, sw[0]
    if (K | N | E) > _I32_MAX:
        _too_wide(fn)
    group = _check_w4(fn, w_codes, w_scales, zeros, (E, N), K)
    _check_rows(fn, M, E, offsets, row_index, row_div)
    t_s, t_out = _float(w_scales), _float(out)
    dev, (pa, pw, ps, pz, po, pout, pi) = _arrays(fn, (a, w_codes, w_scales, zeros, offsets, out, row_index))
    _run(fn, _lib.moe_w4_grouped_gemm, dev, stream, pa, rows, pi, row_div, pw, t_s, ps, pz, group, M, K, N, E,
         po, t_out, pout)


# ---------------------------------------------------------------- device plumbing
def moe_hbm_read(buf, sink, stream=None):
    """Streaming read of every byte of buf (device, 16-byte aligned, size a
    multiple of 16); sink: a one-word device tensor the kernel may write."""
    _check("moe_hbm_read", _lib.moe_hbm_read(_ptr(buf), buf.numel() * buf.element_size(),
                                             _ptr(sink), _stream(stream)))


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A device byte buffer (256-byte aligned by the caching allocator)."""
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def to_device_bf16(bits, device="cuda") -> torch.Tensor:
    """bf16 values given as their uint16 bit patterns (numpy) -> bf16 device tensor."""
    import numpy as np
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(device).view(torch.bfloat16)


def experts_to_device(host: dict, device="cuda", qmode: int = MOE_QMODE_W) -> ExpertWeights:
    """Expert weights as stored on the host (numpy) -> ExpertWeights on the device."""
    import numpy as np
    dt = DTYPE_NAMES[host["dtype"]]

    def dev(key):
        a = host.get(key)
        if a is None:
            return None
        if a.dtype == np.uint16:
            return to_device_bf16(a, device)
        return torch.from_numpy(np.ascontiguousarray(a)).to(device)

    return ExpertWeights(dt, dev("gate_up"), dev("down"), dev("gate_up_scale"), dev("down_scale"),
                         dev("gate_up_gscale"), dev("down_gscale"), qmode)
