"""Python binding of libfalqon.so, the gfx950 HIP library of FALQON's melded
FP8 LoRA linear step.

Argument marshalling only: every function takes device tensors, checks
dtype/shape/contiguity, passes their device pointers and sizes to the C
function of the same name (include/falqon.h) and raises FalqError on a
non-zero status.  All computation runs in the library's HIP kernels on the
stream given (default: torch's current stream).  There is no fallback: if
the library is missing, load() raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from array import array
from typing import Optional

import torch

__all__ = ["load", "FalqError", "fp8_quantize", "fp8_quantize_workspace_bytes",
           "melded_linear_fwd", "melded_linear_bwd", "melded_linear_bwd_workspace_bytes",
           "adapter_step", "adapter_step_adamw", "adamw_state", "ADAMW_STATE_BYTES",
           "rowwise_proxy_update", "rowwise_proxy_update_topk_rank",
           "rowwise_proxy_update_topk_rank_workspace_bytes",
           "fp8_dequantize", "melded_linear_fwd_frozen_a", "fp8_quantize_fmt",
           "melded_linear_bwd_fmt", "melded_linear_bwd_frozen_a_fmt", "FORMATS",
           "melded_linear_fwd_frozen_a_workspace_bytes", "melded_linear_bwd_frozen_a",
           "melded_linear_bwd_frozen_a_workspace_bytes", "rowwise_proxy_update_workspace_bytes",
           "fp4_quantize", "melded_linear_fwd_fp4", "version", "LIB_PATH",
           "fp8_quantize_noalloc", "QUANTIZE_SCRATCH_BYTES", "fp8_quantize_wait_ticks",
           "melded_linear_xa_fused", "melded_linear_fwd_xa", "melded_linear_bwd_xa",
           "melded_linear_bwd_xa_t", "rowwise_proxy_update_t", "fp8_transpose",
           "adapter_pieces_bytes", "adapter_pieces", "adapter_step_pieces",
           "melded_linear_fwd_xa_pieces",
           "melded_linear_fwd_xa_workspace_bytes", "melded_linear_bwd_xa_workspace_bytes",
           "lora_separate_fp8_saved_bytes", "lora_separate_fp8_workspace_bytes",
           "lora_separate_fp8_fwd", "lora_separate_fp8_bwd", "lora_bf16_saved_bytes",
           "lora_bf16_workspace_bytes", "lora_bf16_fwd", "lora_bf16_bwd", "layer_norm_fwd",
           "layer_norm_bwd", "layer_norm_bwd_workspace_bytes", "ACTIVATIONS",
           "melded_linear_fwd_act", "melded_linear_fwd_act_workspace_bytes",
           "linear_act_bwd", "linear_act_bwd_workspace_bytes",
           "grad_norm", "grad_clip", "grad_norm_workspace_bytes", "GRAD_MAX_TENSORS",
           "mxfp4_scales_shape", "mxfp4_scale_bytes", "mxfp4_quantize", "mxfp4_dequantize", "melded_linear_fwd_mxfp4",
           "melded_linear_fwd_mxfp4_workspace_bytes", "checkpoint_scales_shape",
           "checkpoint_save", "checkpoint_restore", "linear_act_bwd_ckpt", "layer_norm_bwd_ckpt",
           "linear_cross_entropy_fwd", "linear_cross_entropy_fwd_workspace_bytes",
           "linear_cross_entropy_bwd", "linear_cross_entropy_bwd_workspace_bytes"]

#: bytes of the per-device scratch array behind fp8_quantize_noalloc
QUANTIZE_SCRATCH_BYTES = 16384

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfalqon.so")
_lib = None

_c_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t
_f32 = ctypes.c_float
_i32 = ctypes.c_int

_SIGS = {
    "falq_status_string": (ctypes.c_char_p, [_i32]),
    "falq_version": (ctypes.c_char_p, []),
    "fp8_quantize_workspace_bytes": (_sz, [_i64]),
    "fp8_quantize": (_i32, [_c_p, _i32, _i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _sz, _c_p]),
    "melded_linear_fwd": (_i32, [_c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64, _c_p, _c_p]),
    "melded_linear_bwd_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "melded_linear_bwd": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _i64, _i64,
                                 _i64, _i64, _c_p, _c_p, _c_p, _c_p, _sz, _c_p]),
    "adapter_step": (_i32, [_c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64, _f32, _c_p]),
    "adapter_step_adamw": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _i64, _i64,
                                  _i64, _f32, _f32, _f32, _f32, _f32, _c_p, _c_p]),
    "fp8_dequantize": (_i32, [_c_p, _c_p, _i64, _c_p, _c_p]),
    "fp8_transpose": (_i32, [_c_p, _i64, _i64, _c_p, _c_p]),
    "fp8_quantize_fmt": (_i32, [_c_p, _i32, _i64, _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _sz,
                                _c_p]),
    "melded_linear_bwd_fmt": (_i32, [_c_p, _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _i64,
                                     _i64, _i64, _i64, _c_p, _c_p, _c_p, _c_p, _sz, _c_p]),
    "melded_linear_bwd_frozen_a_fmt": (_i32, [_c_p, _i32, _c_p, _c_p, _c_p, _c_p, _i64, _i64,
                                              _i64, _i64, _c_p, _c_p, _c_p, _sz, _c_p]),
    "melded_linear_fwd_frozen_a_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "melded_linear_fwd_frozen_a": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64,
                                          _i64, _c_p, _c_p, _c_p, _sz, _c_p]),
    "melded_linear_bwd_frozen_a_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "melded_linear_bwd_frozen_a": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64, _i64,
                                          _c_p, _c_p, _c_p, _sz, _c_p]),
    "rowwise_proxy_update_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "rowwise_proxy_update_topk_rank_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "rowwise_proxy_update_topk_rank": (_i32, [_c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64, _i64,
                                              _f32, _i64, _c_p, _c_p, _c_p, _c_p, _c_p, _sz,
                                              _c_p]),
    "rowwise_proxy_update": (_i32, [_c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64, _f32, _i64, _c_p,
                                    _c_p, _c_p, _c_p, _sz, _c_p]),
    "rowwise_proxy_update_t": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64, _f32, _i64,
                                      _c_p, _c_p, _c_p, _c_p, _sz, _c_p]),
    "fp4_quantize": (_i32, [_c_p, _i32, _i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _sz, _c_p]),
    "fp8_quantize_wait_ticks": (ctypes.c_uint64, [ctypes.c_uint64]),
    "fp8_quantize_noalloc": (_i32, [_c_p, _i32, _i64, _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "melded_linear_fwd_fp4": (_i32, [_c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64, _c_p, _c_p]),
    "melded_linear_xa_fused": (_i32, [_i64, _i64, _i64, _i64]),
    "adapter_pieces_bytes": (_sz, [_i64, _i64]),
    "adapter_pieces": (_i32, [_c_p, _i64, _i64, _c_p, _sz, _c_p]),
    "adapter_step_pieces": (_i32, [_c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64, _f32, _c_p, _sz,
                                   _c_p]),
    "melded_linear_fwd_xa_pieces": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _sz, _i64, _i64, _i64,
                                           _i64, _c_p, _c_p, _c_p]),
    "melded_linear_fwd_xa_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "melded_linear_fwd_xa": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64, _i64, _c_p,
                                    _c_p, _c_p, _sz, _c_p]),
    "melded_linear_bwd_xa_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "melded_linear_bwd_xa": (_i32, [_c_p, _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                    _i64, _i64, _i64, _i64, _c_p, _c_p, _c_p, _c_p, _sz, _c_p]),
    "melded_linear_bwd_xa_t": (_i32, [_c_p, _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                      _i64, _i64, _i64, _i64, _c_p, _c_p, _c_p, _c_p, _sz, _c_p]),
    "lora_separate_fp8_saved_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "lora_separate_fp8_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "lora_separate_fp8_fwd": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64, _i64,
                                     _c_p, _c_p, _sz, _c_p, _sz, _c_p]),
    "lora_separate_fp8_bwd": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _sz, _i64, _i64,
                                     _i64, _i64, _c_p, _c_p, _c_p, _c_p, _sz, _c_p]),
    "lora_bf16_saved_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "lora_bf16_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "lora_bf16_fwd": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64, _i64,
                             _c_p, _c_p, _sz, _c_p, _sz, _c_p]),
    "lora_bf16_bwd": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _sz, _i64,
                             _i64, _i64, _i64, _c_p, _c_p, _c_p, _c_p, _sz, _c_p]),
    "layer_norm_fwd": (_i32, [_c_p, _i32, _c_p, _c_p, _i64, _i64, _f32, _c_p, _i32, _c_p, _c_p,
                              _c_p]),
    "layer_norm_bwd_workspace_bytes": (_sz, [_i64, _i64]),
    "layer_norm_bwd": (_i32, [_c_p, _i32, _c_p, _i32, _c_p, _c_p, _c_p, _i64, _i64, _c_p, _c_p,
                              _c_p, _c_p, _sz, _c_p]),
    "melded_linear_fwd_act_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "melded_linear_fwd_act": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _i32, _c_p, _i64, _i64, _i64,
                                     _i32, _c_p, _c_p, _c_p, _sz, _c_p]),
    "linear_act_bwd_workspace_bytes": (_sz, [_i64, _i64]),
    "linear_act_bwd": (_i32, [_c_p, _i32, _c_p, _i32, _i32, _i64, _i64, _c_p, _c_p, _c_p, _sz,
                              _c_p]),
    "mxfp4_scale_bytes": (_sz, [_i64, _i64]),
    "mxfp4_quantize": (_i32, [_c_p, _i32, _i64, _i64, _c_p, _c_p, _c_p]),
    "mxfp4_dequantize": (_i32, [_c_p, _c_p, _i64, _i64, _c_p, _i32, _c_p]),
    "melded_linear_fwd_mxfp4_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "melded_linear_fwd_mxfp4": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _i32, _c_p, _i64, _i64, _i64,
                                       _i32, _c_p, _c_p, _c_p, _sz, _c_p]),
    "checkpoint_save": (_i32, [_c_p, _i32, _i64, _i64, _c_p, _c_p, _c_p]),
    "checkpoint_restore": (_i32, [_c_p, _c_p, _i64, _i64, _c_p, _i32, _c_p]),
    "linear_act_bwd_ckpt": (_i32, [_c_p, _i32, _c_p, _c_p, _i32, _i64, _i64, _c_p, _c_p, _c_p,
                                   _sz, _c_p]),
    "layer_norm_bwd_ckpt": (_i32, [_c_p, _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _i64, _i64, _c_p,
                                   _c_p, _c_p, _c_p, _sz, _c_p]),
    "linear_cross_entropy_fwd_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "linear_cross_entropy_fwd": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _i64, _i64, _i64, _c_p,
                                        _c_p, _c_p, _sz, _c_p]),
    "linear_cross_entropy_bwd_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32]),
    "linear_cross_entropy_bwd": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _i64, _i64,
                                        _i64, _c_p, _i32, _c_p, _sz, _c_p]),
    "grad_norm_workspace_bytes": (_sz, [_i64]),
    "grad_norm": (_i32, [_i64, _c_p, _c_p, _c_p, _c_p, _c_p, _sz, _c_p]),
    "grad_clip": (_i32, [_i64, _c_p, _c_p, _c_p, _f32, _f32, _c_p, _c_p, _c_p, _sz, _c_p]),
}


class FalqError(RuntimeError):
    pass


#: FP8 code formats (falq_fp8_format): OCP E4M3 and OCP E5M2
FORMATS = {"e4m3": 0, "e5m2": 1}


def _fmt(f) -> int:
    if f not in FORMATS:
        raise FalqError(f"format must be one of {sorted(FORMATS)}, not {f!r}")
    return FORMATS[f]


def load(path: Optional[str] = None):
    """Load libfalqon.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise FalqError(f"{p} not found: build it with `python -c 'import __graft_entry__ as g; "
                        f"g.build()'` or `python fp8_quantized_lora_amd/build.py`")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def version() -> str:
    return load().falq_version().decode()


def _check(status: int, what: str):
    if status != 0:
        msg = load().falq_status_string(status).decode()
        raise FalqError(f"{what}: {msg}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise FalqError("tensor arguments must live on the GPU")
    if not t.is_contiguous():
        raise FalqError("tensor arguments must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _req(t: torch.Tensor, dtype, shape, name):
    if t.dtype != dtype:
        raise FalqError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise FalqError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


# ---------------------------------------------------------------------------
def fp8_quantize_workspace_bytes(n: int) -> int:
    return int(load().fp8_quantize_workspace_bytes(n))


def fp8_quantize(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor,
                 scale_in: Optional[torch.Tensor] = None, amax: Optional[torch.Tensor] = None,
                 nonfinite: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                 stream=None, fmt: str = "e4m3") -> None:
    """q = FP8(x * s), s = max / amax(x); fmt "e4m3" (fp8_quantize) or "e5m2"
    (fp8_quantize_fmt)."""
    lib = load()
    if x.dtype == torch.float32:
        dt = 0
    elif x.dtype == torch.bfloat16:
        dt = 1
    else:
        raise FalqError("fp8_quantize: x must be float32 or bfloat16")
    n = x.numel()
    _req(q, torch.uint8, x.shape, "q")
    wsb = fp8_quantize_workspace_bytes(n)
    if ws is None:
        ws = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    f = _fmt(fmt)
    if f == 0:
        _check(lib.fp8_quantize(_ptr(x), dt, n, _ptr(scale_in), _ptr(q), _ptr(scale), _ptr(amax),
                                _ptr(nonfinite), _ptr(ws), ws.numel(), _stream(stream)),
               "fp8_quantize")
    else:
        _check(lib.fp8_quantize_fmt(_ptr(x), dt, n, f, _ptr(scale_in), _ptr(q), _ptr(scale),
                                    _ptr(amax), _ptr(nonfinite), _ptr(ws), ws.numel(),
                                    _stream(stream)), "fp8_quantize_fmt")


def fp8_quantize_fmt(x, q, scale, fmt: str, **kw) -> None:
    fp8_quantize(x, q, scale, fmt=fmt, **kw)


def fp8_quantize_noalloc(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor,
                         scale_in: Optional[torch.Tensor] = None,
                         amax: Optional[torch.Tensor] = None,
                         nonfinite: Optional[torch.Tensor] = None, stream=None,
                         fmt: str = "e4m3") -> None:
    """fp8_quantize with no workspace: the library's per-device scratch array
    holds the amax partials (for callers that cannot allocate).  Calls that
    overlap on one GPU race on that array."""
    if x.dtype == torch.float32:
        dt = 0
    elif x.dtype == torch.bfloat16:
        dt = 1
    else:
        raise FalqError("fp8_quantize_noalloc: x must be float32 or bfloat16")
    _req(q, torch.uint8, x.shape, "q")
    _check(load().fp8_quantize_noalloc(_ptr(x), dt, x.numel(), _fmt(fmt), _ptr(scale_in),
                                       _ptr(q), _ptr(scale), _ptr(amax), _ptr(nonfinite),
                                       _stream(stream)), "fp8_quantize_noalloc")


def fp8_quantize_wait_ticks(ticks: int) -> int:
    """Set how long (100 MHz GPU counter ticks) the one-launch quantize waits
    for the other workgroups' maxima before reading their ranges itself;
    returns the previous setting."""
    if ticks < 0:
        raise FalqError("fp8_quantize_wait_ticks: ticks must be >= 0")
    return int(load().fp8_quantize_wait_ticks(int(ticks)))


def melded_linear_fwd(xq: torch.Tensor, s_x: torch.Tensor, wq: torch.Tensor, s_w: torch.Tensor,
                      y: torch.Tensor, stream=None) -> None:
    T, d_in = xq.shape
    d_out = wq.shape[0]
    _req(wq, torch.uint8, (d_out, d_in), "wq")
    _req(y, torch.float32, (T, d_out), "y")
    _check(load().melded_linear_fwd(_ptr(xq), _ptr(s_x), _ptr(wq), _ptr(s_w), T, d_in, d_out,
                                    _ptr(y), _stream(stream)), "melded_linear_fwd")


def fp4_quantize(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor,
                 scale_in: Optional[torch.Tensor] = None, amax: Optional[torch.Tensor] = None,
                 nonfinite: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    """q = FP4 E2M1(x * s), s = 6 / amax(x), two codes per byte along the last
    axis (q has the shape of x with the last axis halved)."""
    lib = load()
    if x.dtype == torch.float32:
        dt = 0
    elif x.dtype == torch.bfloat16:
        dt = 1
    else:
        raise FalqError("fp4_quantize: x must be float32 or bfloat16")
    if x.dim() == 0 or x.shape[-1] % 2:
        raise FalqError("fp4_quantize: the last axis of x must have even length")
    n = x.numel()
    _req(q, torch.uint8, tuple(x.shape[:-1]) + (x.shape[-1] // 2,), "q")
    wsb = fp8_quantize_workspace_bytes(n)
    if ws is None:
        ws = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    _check(lib.fp4_quantize(_ptr(x), dt, n, _ptr(scale_in), _ptr(q), _ptr(scale), _ptr(amax),
                            _ptr(nonfinite), _ptr(ws), ws.numel(), _stream(stream)),
           "fp4_quantize")


def melded_linear_fwd_fp4(xq: torch.Tensor, s_x: torch.Tensor, wq: torch.Tensor,
                          s_w: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """y = dec(xq) dec(wq)^T / (s_x s_w) with FP4 E2M1 operands (two codes per
    byte: xq [T x d_in/2], wq [d_out x d_in/2])."""
    T, half = xq.shape
    d_in = 2 * half
    d_out = wq.shape[0]
    _req(wq, torch.uint8, (d_out, half), "wq")
    _req(y, torch.float32, (T, d_out), "y")
    _check(load().melded_linear_fwd_fp4(_ptr(xq), _ptr(s_x), _ptr(wq), _ptr(s_w), T, d_in, d_out,
                                        _ptr(y), _stream(stream)), "melded_linear_fwd_fp4")


def melded_linear_bwd_workspace_bytes(T: int, d_in: int, d_out: int, r: int) -> int:
    return int(load().melded_linear_bwd_workspace_bytes(T, d_in, d_out, r))


def melded_linear_bwd(gq, s_g, xq, s_x, wq, s_w, A, B, dx, dA, dB, ws=None, stream=None,
                      g_fmt: str = "e4m3") -> None:
    T, d_out = gq.shape
    d_in = xq.shape[1]
    r = A.shape[0]
    _req(xq, torch.uint8, (T, d_in), "xq")
    _req(wq, torch.uint8, (d_out, d_in), "wq")
    _req(A, torch.float32, (r, d_in), "A")
    _req(B, torch.float32, (d_out, r), "B")
    _req(dB, torch.float32, (d_out, r), "dB")
    if dx is not None:
        _req(dx, torch.float32, (T, d_in), "dx")
    if dA is not None:
        _req(dA, torch.float32, (r, d_in), "dA")
    wsb = melded_linear_bwd_workspace_bytes(T, d_in, d_out, r)
    if ws is None:
        ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=gq.device)
    _check(load().melded_linear_bwd_fmt(_ptr(gq), _fmt(g_fmt), _ptr(s_g), _ptr(xq), _ptr(s_x),
                                        _ptr(wq), _ptr(s_w), _ptr(A), _ptr(B), T, d_in, d_out, r,
                                        _ptr(dx), _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(),
                                        _stream(stream)), "melded_linear_bwd")


def melded_linear_bwd_fmt(gq, g_fmt: str, s_g, xq, s_x, wq, s_w, A, B, dx, dA, dB, **kw) -> None:
    melded_linear_bwd(gq, s_g, xq, s_x, wq, s_w, A, B, dx, dA, dB, g_fmt=g_fmt, **kw)


def fp8_dequantize(q: torch.Tensor, scale: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """out = dec(q) / scale (float32), elementwise."""
    _req(q, torch.uint8, tuple(q.shape), "q")
    _req(out, torch.float32, tuple(q.shape), "out")
    _req(scale, torch.float32, (1,), "scale")
    _check(load().fp8_dequantize(_ptr(q), _ptr(scale), q.numel(), _ptr(out), _stream(stream)),
           "fp8_dequantize")


def melded_linear_fwd_frozen_a_workspace_bytes(T: int, d_in: int, r: int) -> int:
    return int(load().melded_linear_fwd_frozen_a_workspace_bytes(T, d_in, r))


def melded_linear_fwd_frozen_a(xq, s_x, wq, s_w, aq, s_a, y, u, ws=None, stream=None) -> None:
    """y = X~ W~^T / (s_x s_w) and u = X~ A~^T / (s_x s_a)."""
    T, d_in = xq.shape
    d_out = wq.shape[0]
    r = aq.shape[0]
    _req(xq, torch.uint8, (T, d_in), "xq")
    _req(wq, torch.uint8, (d_out, d_in), "wq")
    _req(aq, torch.uint8, (r, d_in), "aq")
    _req(y, torch.float32, (T, d_out), "y")
    _req(u, torch.float32, (T, r), "u")
    need = melded_linear_fwd_frozen_a_workspace_bytes(T, d_in, r)
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=xq.device)
    _check(load().melded_linear_fwd_frozen_a(_ptr(xq), _ptr(s_x), _ptr(wq), _ptr(s_w), _ptr(aq),
                                             _ptr(s_a), T, d_in, d_out, r, _ptr(y), _ptr(u),
                                             _ptr(ws), ws.numel(), _stream(stream)),
           "melded_linear_fwd_frozen_a")


def melded_linear_bwd_frozen_a_workspace_bytes(T: int, d_in: int, d_out: int, r: int) -> int:
    return int(load().melded_linear_bwd_frozen_a_workspace_bytes(T, d_in, d_out, r))


def melded_linear_bwd_frozen_a(gq, s_g, wq, s_w, u, dx, dB, ws=None, stream=None,
                               g_fmt: str = "e4m3") -> None:
    """dx = G~ W~ / (s_g s_w) (dx may be None) and dB = G^^T u."""
    T, d_out = gq.shape
    d_in = wq.shape[1]
    r = u.shape[1]
    _req(gq, torch.uint8, (T, d_out), "gq")
    _req(wq, torch.uint8, (d_out, d_in), "wq")
    _req(u, torch.float32, (T, r), "u")
    _req(dB, torch.float32, (d_out, r), "dB")
    if dx is not None:
        _req(dx, torch.float32, (T, d_in), "dx")
    need = melded_linear_bwd_frozen_a_workspace_bytes(T, d_in, d_out, r)
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=gq.device)
    _check(load().melded_linear_bwd_frozen_a_fmt(_ptr(gq), _fmt(g_fmt), _ptr(s_g), _ptr(wq),
                                                 _ptr(s_w), _ptr(u), T, d_in, d_out, r, _ptr(dx),
                                                 _ptr(dB), _ptr(ws), ws.numel(), _stream(stream)),
           "melded_linear_bwd_frozen_a")


def melded_linear_bwd_frozen_a_fmt(gq, g_fmt: str, s_g, wq, s_w, u, dx, dB, **kw) -> None:
    melded_linear_bwd_frozen_a(gq, s_g, wq, s_w, u, dx, dB, g_fmt=g_fmt, **kw)


def adapter_step(A, B, dA, dB, lr: float, stream=None) -> None:
    r, d_in = A.shape
    d_out = B.shape[0]
    _req(B, torch.float32, (d_out, r), "B")
    _req(dB, torch.float32, (d_out, r), "dB")
    if dA is not None:
        _req(dA, torch.float32, (r, d_in), "dA")
    _check(load().adapter_step(_ptr(A), _ptr(B), _ptr(dA), _ptr(dB), r, d_in, d_out, lr,
                               _stream(stream)), "adapter_step")


#: bytes of the AdamW optimizer state (zero-filled before the first step)
ADAMW_STATE_BYTES = 64


def adamw_state(device="cuda") -> torch.Tensor:
    """A fresh AdamW state: zeros, before step 1 (int64 step count first)."""
    return torch.zeros(ADAMW_STATE_BYTES // 8, dtype=torch.int64, device=device)


def adapter_step_adamw(A, B, dA, dB, mA, vA, mB, vB, state, lr: float, beta1: float = 0.9,
                       beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
                       stream=None) -> None:
    """One AdamW step on A and B with moments mA, vA, mB, vB, in place; `state`
    (adamw_state()) carries the step count and is advanced by the call.  dA =
    None freezes A (mA and vA may then be None)."""
    r, d_in = A.shape
    d_out = B.shape[0]
    for t, name in ((B, "B"), (dB, "dB"), (mB, "mB"), (vB, "vB")):
        _req(t, torch.float32, (d_out, r), name)
    if dA is not None:
        for t, name in ((A, "A"), (dA, "dA"), (mA, "mA"), (vA, "vA")):
            _req(t, torch.float32, (r, d_in), name)
    if state.numel() * state.element_size() != ADAMW_STATE_BYTES:
        raise FalqError(f"state must be {ADAMW_STATE_BYTES} bytes (adamw_state())")
    _check(load().adapter_step_adamw(_ptr(A), _ptr(B), _ptr(dA), _ptr(dB), _ptr(mA), _ptr(vA),
                                     _ptr(mB), _ptr(vB), r, d_in, d_out, lr, beta1, beta2, eps,
                                     weight_decay, _ptr(state), _stream(stream)),
           "adapter_step_adamw")


def rowwise_proxy_update_workspace_bytes(d_in: int, d_out: int, r: int) -> int:
    return int(load().rowwise_proxy_update_workspace_bytes(d_in, d_out, r))


def rowwise_proxy_update_t(wq, wqT, s_w, A, B, tau: float, k_max: int, sel_idx, n_sel, rho=None,
                           ws=None, stream=None) -> None:
    """rowwise_proxy_update that also writes wqT = the updated wq, transposed."""
    d_out, d_in = wq.shape
    r = A.shape[0]
    _req(wqT, torch.uint8, (d_in, d_out), "wqT")
    _req(A, torch.float32, (r, d_in), "A")
    _req(B, torch.float32, (d_out, r), "B")
    _req(sel_idx, torch.int32, (d_out,), "sel_idx")
    if rho is not None:
        _req(rho, torch.float32, (d_out,), "rho")
    wsb = rowwise_proxy_update_workspace_bytes(d_in, d_out, r)
    if ws is None:
        ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=wq.device)
    _check(load().rowwise_proxy_update_t(_ptr(wq), _ptr(wqT), _ptr(s_w), _ptr(A), _ptr(B), d_in,
                                         d_out, r, tau, k_max, _ptr(sel_idx), _ptr(n_sel),
                                         _ptr(rho), _ptr(ws), ws.numel(), _stream(stream)),
           "rowwise_proxy_update_t")


def rowwise_proxy_update(wq, s_w, A, B, tau: float, k_max: int, sel_idx, n_sel, rho=None, ws=None,
                         stream=None) -> None:
    d_out, d_in = wq.shape
    r = A.shape[0]
    _req(A, torch.float32, (r, d_in), "A")
    _req(B, torch.float32, (d_out, r), "B")
    _req(sel_idx, torch.int32, (d_out,), "sel_idx")
    if rho is not None:
        _req(rho, torch.float32, (d_out,), "rho")
    wsb = rowwise_proxy_update_workspace_bytes(d_in, d_out, r)
    if ws is None:
        ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=wq.device)
    _check(load().rowwise_proxy_update(_ptr(wq), _ptr(s_w), _ptr(A), _ptr(B), d_in, d_out, r, tau,
                                       k_max, _ptr(sel_idx), _ptr(n_sel), _ptr(rho), _ptr(ws),
                                       ws.numel(), _stream(stream)), "rowwise_proxy_update")




def rowwise_proxy_update_topk_rank_workspace_bytes(d_in: int, d_out: int, r: int,
                                                   k_rank: int) -> int:
    return int(load().rowwise_proxy_update_topk_rank_workspace_bytes(d_in, d_out, r, k_rank))


def rowwise_proxy_update_topk_rank(wq, s_w, A, B, k_rank: int, tau: float, k_max: int, sel_idx,
                                   n_sel, comp_idx, rho=None, ws=None, stream=None) -> None:
    """The row-wise proxy update over the k_rank rank components of largest
    score (comp_idx receives them, ascending)."""
    d_out, d_in = wq.shape
    r = A.shape[0]
    _req(A, torch.float32, (r, d_in), "A")
    _req(B, torch.float32, (d_out, r), "B")
    _req(comp_idx, torch.int32, (k_rank,), "comp_idx")
    need = rowwise_proxy_update_topk_rank_workspace_bytes(d_in, d_out, r, k_rank)
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=wq.device)
    _check(load().rowwise_proxy_update_topk_rank(
        _ptr(wq), _ptr(s_w), _ptr(A), _ptr(B), d_in, d_out, r, k_rank, tau, k_max, _ptr(sel_idx),
        _ptr(n_sel), _ptr(rho), _ptr(comp_idx), _ptr(ws), ws.numel(), _stream(stream)),
        "rowwise_proxy_update_topk_rank")


# ---------------------------------------------------------------------------
# X^ A^T formed with the forward product, G^ B with the dX product
def melded_linear_xa_fused(T: int, d_in: int, d_out: int, r: int) -> bool:
    """Whether X^ A^T and G^ B ride in the FP8 products for this shape."""
    return bool(load().melded_linear_xa_fused(T, d_in, d_out, r))


def melded_linear_fwd_xa_workspace_bytes(T: int, d_in: int, d_out: int, r: int) -> int:
    return int(load().melded_linear_fwd_xa_workspace_bytes(T, d_in, d_out, r))


def melded_linear_bwd_xa_workspace_bytes(T: int, d_in: int, d_out: int, r: int) -> int:
    return int(load().melded_linear_bwd_xa_workspace_bytes(T, d_in, d_out, r))


def melded_linear_fwd_xa(xq, s_x, wq, s_w, A, y, xa, ws=None, stream=None) -> None:
    """y = X~ W~^T / (s_x s_w) and xa = X^ A^T (the factor dB needs)."""
    T, d_in = xq.shape
    d_out = wq.shape[0]
    r = A.shape[0]
    _req(wq, torch.uint8, (d_out, d_in), "wq")
    _req(A, torch.float32, (r, d_in), "A")
    _req(y, torch.float32, (T, d_out), "y")
    _req(xa, torch.float32, (T, r), "xa")
    ws = _buf(ws, melded_linear_fwd_xa_workspace_bytes(T, d_in, d_out, r), xq.device, "ws")
    _check(load().melded_linear_fwd_xa(_ptr(xq), _ptr(s_x), _ptr(wq), _ptr(s_w), _ptr(A), T, d_in,
                                       d_out, r, _ptr(y), _ptr(xa), _ptr(ws), ws.numel(),
                                       _stream(stream)), "melded_linear_fwd_xa")


def adapter_pieces_bytes(r: int, d_in: int) -> int:
    """Bytes of the buffer that holds A's pieces (0: not available)."""
    return int(load().adapter_pieces_bytes(r, d_in))


def adapter_pieces(A, pieces, stream=None) -> None:
    """A's block-scaled E4M3 pieces into `pieces` (uint8, adapter_pieces_bytes)."""
    r, d_in = A.shape
    _req(A, torch.float32, (r, d_in), "A")
    _check(load().adapter_pieces(_ptr(A), r, d_in, _ptr(pieces), pieces.numel(),
                                 _stream(stream)), "adapter_pieces")


def adapter_step_pieces(A, B, dA, dB, lr: float, pieces, stream=None) -> None:
    """adapter_step (SGD on A and B), and the pieces of the new A into `pieces`."""
    r, d_in = A.shape
    d_out = B.shape[0]
    _req(A, torch.float32, (r, d_in), "A")
    _req(dA, torch.float32, (r, d_in), "dA")
    _req(B, torch.float32, (d_out, r), "B")
    _req(dB, torch.float32, (d_out, r), "dB")
    _check(load().adapter_step_pieces(_ptr(A), _ptr(B), _ptr(dA), _ptr(dB), r, d_in, d_out, lr,
                                      _ptr(pieces), pieces.numel(), _stream(stream)),
           "adapter_step_pieces")


def melded_linear_fwd_xa_pieces(xq, s_x, wq, s_w, pieces, r: int, y, xa, stream=None) -> None:
    """melded_linear_fwd_xa with A given as its pieces (adapter_pieces / adapter_step_pieces)."""
    T, d_in = xq.shape
    d_out = wq.shape[0]
    _req(wq, torch.uint8, (d_out, d_in), "wq")
    _req(y, torch.float32, (T, d_out), "y")
    _req(xa, torch.float32, (T, r), "xa")
    _check(load().melded_linear_fwd_xa_pieces(_ptr(xq), _ptr(s_x), _ptr(wq), _ptr(s_w),
                                              _ptr(pieces), pieces.numel(), T, d_in, d_out, r,
                                              _ptr(y), _ptr(xa), _stream(stream)),
           "melded_linear_fwd_xa_pieces")


def melded_linear_bwd_xa(gq, s_g, xq, s_x, wq, s_w, A, B, xa, dx, dA, dB, ws=None, stream=None,
                         g_fmt: str = "e4m3", wq_t: bool = False) -> None:
    """dx, dA = (G^ B)^T X^ and dB = G^^T xa, with xa from melded_linear_fwd_xa.
    wq_t: wq is the backbone's transpose [d_in x d_out] (melded_linear_bwd_xa_t)."""
    T, d_out = gq.shape
    d_in = xq.shape[1]
    r = A.shape[0]
    _req(wq, torch.uint8, (d_in, d_out) if wq_t else (d_out, d_in), "wqT" if wq_t else "wq")
    _req(A, torch.float32, (r, d_in), "A")
    _req(B, torch.float32, (d_out, r), "B")
    _req(xa, torch.float32, (T, r), "xa")
    _req(dB, torch.float32, (d_out, r), "dB")
    if dx is not None:
        _req(dx, torch.float32, (T, d_in), "dx")
    if dA is not None:
        _req(dA, torch.float32, (r, d_in), "dA")
    ws = _buf(ws, melded_linear_bwd_xa_workspace_bytes(T, d_in, d_out, r), gq.device, "ws")
    name = "melded_linear_bwd_xa_t" if wq_t else "melded_linear_bwd_xa"
    _check(getattr(load(), name)(_ptr(gq), _fmt(g_fmt), _ptr(s_g), _ptr(xq), _ptr(s_x),
                                 _ptr(wq), _ptr(s_w), _ptr(A), _ptr(B), _ptr(xa), T, d_in,
                                 d_out, r, _ptr(dx), _ptr(dA), _ptr(dB), _ptr(ws),
                                 ws.numel(), _stream(stream)), name)


def melded_linear_bwd_xa_t(gq, s_g, xq, s_x, wqT, s_w, A, B, xa, dx, dA, dB, ws=None,
                           stream=None, g_fmt: str = "e4m3") -> None:
    """melded_linear_bwd_xa with the backbone handed in transposed, wqT [d_in x d_out]."""
    melded_linear_bwd_xa(gq, s_g, xq, s_x, wqT, s_w, A, B, xa, dx, dA, dB, ws=ws, stream=stream,
                         g_fmt=g_fmt, wq_t=True)


def fp8_transpose(q: torch.Tensor, qT: torch.Tensor, stream=None) -> None:
    """qT = q^T for a byte matrix (rows and columns multiples of 16)."""
    rows, cols = q.shape
    _req(q, torch.uint8, (rows, cols), "q")
    _req(qT, torch.uint8, (cols, rows), "qT")
    _check(load().fp8_transpose(_ptr(q), rows, cols, _ptr(qT), _stream(stream)), "fp8_transpose")


# ---------------------------------------------------------------------------
# the baselines: LoRA with a separate adapter branch (separate-path FP8, bf16)
def lora_separate_fp8_saved_bytes(T: int, d_in: int, d_out: int, r: int) -> int:
    return int(load().lora_separate_fp8_saved_bytes(T, d_in, d_out, r))


def lora_separate_fp8_workspace_bytes(T: int, d_in: int, d_out: int, r: int) -> int:
    return int(load().lora_separate_fp8_workspace_bytes(T, d_in, d_out, r))


def lora_bf16_saved_bytes(T: int, d_in: int, d_out: int, r: int) -> int:
    return int(load().lora_bf16_saved_bytes(T, d_in, d_out, r))


def lora_bf16_workspace_bytes(T: int, d_in: int, d_out: int, r: int) -> int:
    return int(load().lora_bf16_workspace_bytes(T, d_in, d_out, r))


def _buf(t, nbytes, device, name):
    if t is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    if t.numel() * t.element_size() < nbytes:
        raise FalqError(f"{name}: needs {nbytes} bytes")
    return t


def lora_separate_fp8_fwd(xq, s_x, wq, s_w, A, B, y, saved, ws=None, stream=None) -> None:
    """Y = X^ W^^T + Q(X^ Q(A)^T)^ Q(B)^^T: the layer with a separate FP8 LoRA
    branch; `saved` (lora_separate_fp8_saved_bytes, uint8) keeps A~, B~, U~
    and their scales for the backward."""
    T, d_in = xq.shape
    d_out = wq.shape[0]
    r = A.shape[0]
    _req(wq, torch.uint8, (d_out, d_in), "wq")
    _req(A, torch.float32, (r, d_in), "A")
    _req(B, torch.float32, (d_out, r), "B")
    _req(y, torch.float32, (T, d_out), "y")
    ws = _buf(ws, lora_separate_fp8_workspace_bytes(T, d_in, d_out, r), xq.device, "ws")
    _check(load().lora_separate_fp8_fwd(_ptr(xq), _ptr(s_x), _ptr(wq), _ptr(s_w), _ptr(A),
                                        _ptr(B), T, d_in, d_out, r, _ptr(y), _ptr(saved),
                                        saved.numel() * saved.element_size(), _ptr(ws),
                                        ws.numel(), _stream(stream)), "lora_separate_fp8_fwd")


def lora_separate_fp8_bwd(gq, s_g, xq, s_x, wq, s_w, saved, r: int, dx, dA, dB, ws=None,
                          stream=None) -> None:
    """dX, dA, dB of the separate-path FP8 LoRA layer from the forward's `saved`."""
    T, d_out = gq.shape
    d_in = xq.shape[1]
    _req(dx, torch.float32, (T, d_in), "dx")
    _req(dA, torch.float32, (r, d_in), "dA")
    _req(dB, torch.float32, (d_out, r), "dB")
    ws = _buf(ws, lora_separate_fp8_workspace_bytes(T, d_in, d_out, r), gq.device, "ws")
    _check(load().lora_separate_fp8_bwd(_ptr(gq), _ptr(s_g), _ptr(xq), _ptr(s_x), _ptr(wq),
                                        _ptr(s_w), _ptr(saved),
                                        saved.numel() * saved.element_size(), T, d_in, d_out, r,
                                        _ptr(dx), _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(),
                                        _stream(stream)), "lora_separate_fp8_bwd")


def lora_bf16_fwd(x, xq, s_x, wq, s_w, A, B, y, saved, ws=None, stream=None) -> None:
    """Y = X^ W^^T + bf(bf(X) bf(A)^T) bf(B)^T: the FP8 backbone with a bf16
    LoRA branch; `saved` (lora_bf16_saved_bytes) keeps bf(U)."""
    T, d_in = xq.shape
    d_out = wq.shape[0]
    r = A.shape[0]
    _req(x, torch.float32, (T, d_in), "x")
    _req(A, torch.float32, (r, d_in), "A")
    _req(B, torch.float32, (d_out, r), "B")
    _req(y, torch.float32, (T, d_out), "y")
    ws = _buf(ws, lora_bf16_workspace_bytes(T, d_in, d_out, r), xq.device, "ws")
    _check(load().lora_bf16_fwd(_ptr(x), _ptr(xq), _ptr(s_x), _ptr(wq), _ptr(s_w), _ptr(A),
                                _ptr(B), T, d_in, d_out, r, _ptr(y), _ptr(saved),
                                saved.numel() * saved.element_size(), _ptr(ws), ws.numel(),
                                _stream(stream)), "lora_bf16_fwd")


def lora_bf16_bwd(dy, gq, s_g, x, wq, s_w, A, B, saved, dx, dA, dB, ws=None,
                  stream=None) -> None:
    """dX, dA, dB of the bf16 LoRA layer from the forward's `saved`."""
    T, d_out = gq.shape
    d_in = x.shape[1]
    r = A.shape[0]
    _req(dy, torch.float32, (T, d_out), "dy")
    _req(dx, torch.float32, (T, d_in), "dx")
    _req(dA, torch.float32, (r, d_in), "dA")
    _req(dB, torch.float32, (d_out, r), "dB")
    ws = _buf(ws, lora_bf16_workspace_bytes(T, d_in, d_out, r), gq.device, "ws")
    _check(load().lora_bf16_bwd(_ptr(dy), _ptr(gq), _ptr(s_g), _ptr(x), _ptr(wq), _ptr(s_w),
                                _ptr(A), _ptr(B), _ptr(saved),
                                saved.numel() * saved.element_size(), T, d_in, d_out, r,
                                _ptr(dx), _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(),
                                _stream(stream)), "lora_bf16_bwd")


# ---------------------------------------------------------------------------
# Around the linear: layer norm, the product with an epilogue, clipping.
# These calls run on the device of their tensors, whichever is current.

#: activations of melded_linear_fwd_act and linear_act_bwd (falq_activation)
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
#: tensors that one grad_norm or grad_clip call takes at most
GRAD_MAX_TENSORS = 65536

_ELEM = {torch.float32: 0, torch.bfloat16: 1}
# (absent from a torch built without a GPU, where every call is refused before
# they are needed)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _elem(t: torch.Tensor, name: str) -> int:
    e = _ELEM.get(t.dtype)
    if e is None:
        raise FalqError(f"{name}: expected float32 or bfloat16, got {t.dtype}")
    return e


def _act(act) -> int:
    if not isinstance(act, str) or act not in ACTIVATIONS:
        raise FalqError(f"act must be one of {sorted(ACTIVATIONS)}, not {act!r}")
    return ACTIVATIONS[act]


def _arg(t: Optional[torch.Tensor], dtype, shape, dev: int, name: str) -> Optional[int]:
    """The address of t (None: not given), a contiguous tensor of that type and
    shape on device dev.  The small calls are bound by the host, so the checks
    take the short way where all hold."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _req(t, dtype, shape, name)
    _ptr(t)
    raise FalqError(f"{name}: expected device cuda:{dev}, got {t.device}")


def _matrix(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise FalqError(f"{name}: expected two dimensions, got shape {tuple(t.shape)}")
    return t.shape


def _device(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise FalqError(f"{name}: tensor arguments must live on the GPU")
    return dev


def _stream_of(dev: int, stream) -> int:
    return _raw_stream(dev) if stream is None else _stream(stream)


def _scratch(ws: Optional[torch.Tensor], need: int, dev: int, stream, st: int):
    """The caller's workspace, or one allocated for the stream of the call, so
    that its memory is not handed to other work while the call runs."""
    if ws is not None:
        if ws.dtype is not torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
            raise FalqError(f"ws must be contiguous uint8 on cuda:{dev}")
        return ws
    if not need:
        return None
    with _on_stream(dev, stream, st):
        return torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", dev))


def _on_stream(dev: int, stream, st: int):
    """A context in which torch's own work is on the call's stream."""
    if stream is None or st == _raw_stream(dev):
        return contextlib.nullcontext()
    where = torch.device("cuda", dev)
    return torch.cuda.stream(torch.cuda.ExternalStream(st, device=where) if st
                             else torch.cuda.default_stream(where))


def _run(fn, what: str, dev: int, *args) -> None:
    if dev == _current_device():
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status:
        _check(status, what)


def layer_norm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor],
                   y: torch.Tensor, mean: Optional[torch.Tensor] = None,
                   rstd: Optional[torch.Tensor] = None, eps: float = 1e-5, stream=None) -> None:
    """y = (x - mean) * rstd * weight + bias per row of x [T x d], rstd =
    1 / sqrt(var + eps); x and y float32 or bfloat16 each, weight and bias
    float32 or None; mean and rstd [T] are what layer_norm_bwd takes."""
    T, d = _matrix(x, "x")
    xt, yt, dev = _elem(x, "x"), _elem(y, "y"), _device(x, "x")
    f32 = torch.float32
    _run(load().layer_norm_fwd, "layer_norm_fwd", dev, _arg(x, x.dtype, (T, d), dev, "x"), xt,
         _arg(weight, f32, (d,), dev, "weight"), _arg(bias, f32, (d,), dev, "bias"), T, d, eps,
         _arg(y, y.dtype, (T, d), dev, "y"), yt, _arg(mean, f32, (T,), dev, "mean"),
         _arg(rstd, f32, (T,), dev, "rstd"), _stream_of(dev, stream))


def layer_norm_bwd_workspace_bytes(T: int, d: int) -> int:
    return int(load().layer_norm_bwd_workspace_bytes(T, d))


def layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor],
                   mean: torch.Tensor, rstd: torch.Tensor, dx: Optional[torch.Tensor],
                   dweight: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """The gradients of layer_norm_fwd: dx (dy's type; may be dy, or None), and
    the sums over rows dweight and dbias (float32, each may be None)."""
    T, d = _matrix(x, "x")
    gt, xt, dev = _elem(dy, "dy"), _elem(x, "x"), _device(x, "x")
    f32, lib, st = torch.float32, load(), _stream_of(dev, stream)
    args = (_arg(dy, dy.dtype, (T, d), dev, "dy"), gt, _arg(x, x.dtype, (T, d), dev, "x"), xt,
            _arg(weight, f32, (d,), dev, "weight"), _arg(mean, f32, (T,), dev, "mean"),
            _arg(rstd, f32, (T,), dev, "rstd"), T, d, _arg(dx, dy.dtype, (T, d), dev, "dx"),
            _arg(dweight, f32, (d,), dev, "dweight"), _arg(dbias, f32, (d,), dev, "dbias"))
    need = (0 if dweight is None and dbias is None
            else lib.layer_norm_bwd_workspace_bytes(T, d))
    w = _scratch(ws, need, dev, stream, st)
    _run(lib.layer_norm_bwd, "layer_norm_bwd", dev, *args, *_span(w), st)


def _span(ws: Optional[torch.Tensor]):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel())


def melded_linear_fwd_act_workspace_bytes(T: int, d_in: int, d_out: int) -> int:
    return int(load().melded_linear_fwd_act_workspace_bytes(T, d_in, d_out))


def melded_linear_fwd_act(xq: torch.Tensor, s_x: torch.Tensor, wq: torch.Tensor,
                          s_w: torch.Tensor, y: torch.Tensor,
                          bias: Optional[torch.Tensor] = None, act: str = "none",
                          residual: Optional[torch.Tensor] = None,
                          z: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    """z = dec(xq) dec(wq)^T / (s_x s_w) + bias and y = act(z) + residual in one
    call; y, z and residual share one type (float32 or bfloat16), bias is
    float32; residual may be y; z (None: not kept) is what linear_act_bwd takes."""
    T, d_in = _matrix(xq, "xq")
    d_out = _matrix(wq, "wq")[0]
    t, a, dev = _elem(y, "y"), _act(act), _device(xq, "xq")
    u8, f32, out = torch.uint8, torch.float32, (T, d_out)
    lib, st = load(), _stream_of(dev, stream)
    args = (_arg(xq, u8, (T, d_in), dev, "xq"), _arg(s_x, f32, (1,), dev, "s_x"),
            _arg(wq, u8, (d_out, d_in), dev, "wq"), _arg(s_w, f32, (1,), dev, "s_w"),
            _arg(bias, f32, (d_out,), dev, "bias"), a,
            _arg(residual, y.dtype, out, dev, "residual"), T, d_in, d_out, t,
            _arg(y, y.dtype, out, dev, "y"), _arg(z, y.dtype, out, dev, "z"))
    # up to 16 tokens need no workspace (and are bound by the host)
    need = 0 if T <= 16 else lib.melded_linear_fwd_act_workspace_bytes(T, d_in, d_out)
    w = _scratch(ws, need, dev, stream, st)
    _run(lib.melded_linear_fwd_act, "melded_linear_fwd_act", dev, *args, *_span(w), st)


def linear_act_bwd_workspace_bytes(T: int, d_out: int) -> int:
    return int(load().linear_act_bwd_workspace_bytes(T, d_out))


def linear_act_bwd(dy: torch.Tensor, z: Optional[torch.Tensor], dz: Optional[torch.Tensor],
                   dbias: Optional[torch.Tensor] = None, act: str = "none",
                   ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """dz = dy * act'(z) (dy's type; dz may be dy) and dbias = the sum of dz over
    the rows (float32); either may be None.  z float32 or bfloat16, None for act
    "none"."""
    T, d_out = _matrix(dy, "dy")
    gt, a = _elem(dy, "dy"), _act(act)
    if z is None and a != 0:
        raise FalqError(f"linear_act_bwd: z is needed for act {act!r}")
    zt = 0 if z is None else _elem(z, "z")
    dev, lib = _device(dy, "dy"), load()
    st = _stream_of(dev, stream)
    args = (_arg(dy, dy.dtype, (T, d_out), dev, "dy"), gt,
            None if z is None else _arg(z, z.dtype, (T, d_out), dev, "z"), zt, a, T, d_out,
            _arg(dz, dy.dtype, (T, d_out), dev, "dz"),
            _arg(dbias, torch.float32, (d_out,), dev, "dbias"))
    need = 0 if dbias is None else lib.linear_act_bwd_workspace_bytes(T, d_out)
    w = _scratch(ws, need, dev, stream, st)
    _run(lib.linear_act_bwd, "linear_act_bwd", dev, *args, *_span(w), st)


def grad_norm_workspace_bytes(count: int) -> int:
    return int(load().grad_norm_workspace_bytes(count))


def _addresses(what: str, tensors, dev: int) -> array:
    """Host array of the tensors' addresses, all contiguous on device dev."""
    for t in tensors:
        if t.get_device() != dev or not t.is_contiguous():
            raise FalqError(f"{what}: every tensor must be contiguous and on cuda:{dev}")
    return array("q", [t.data_ptr() for t in tensors])


def _sizes_types(what: str, tensors):
    try:
        kinds = array("i", [_ELEM[t.dtype] for t in tensors])
    except KeyError as e:
        raise FalqError(f"{what}: expected float32 or bfloat16, got {e.args[0]}") from None
    return array("q", [t.numel() for t in tensors]), kinds


def _at(a: array) -> int:
    return a.buffer_info()[0]


def grad_norm(grads, norm: torch.Tensor, ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """norm = sqrt of the sum of squares over all elements of all tensors
    (float32 and bfloat16, any shapes), summed in float64 on the device."""
    grads, dev, lib = list(grads), _device(norm, "norm"), load()
    st, count = _stream_of(dev, stream), len(grads)
    p, (n, t) = _addresses("grad_norm", grads, dev), _sizes_types("grad_norm", grads)
    out = _arg(norm, torch.float32, (1,), dev, "norm")
    w = _scratch(ws, lib.grad_norm_workspace_bytes(count), dev, stream, st)
    _run(lib.grad_norm, "grad_norm", dev, count, _at(p), _at(n), _at(t), out, *_span(w), st)


def grad_clip(grads, max_norm: float, norm: torch.Tensor, out=None, eps: float = 1e-6,
              ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """Multiply every tensor by min(1, max_norm / (norm + eps)), norm being the
    global norm over all of them (written to `norm` as grad_norm does): in
    place, or into the tensors `out`.  No tensor may be listed twice."""
    grads, dev, lib = list(grads), _device(norm, "norm"), load()
    st, count = _stream_of(dev, stream), len(grads)
    p, (n, t) = _addresses("grad_clip", grads, dev), _sizes_types("grad_clip", grads)
    q = None
    if out is not None:
        out = list(out)
        if len(out) != count:
            raise FalqError(f"grad_clip: {len(out)} outputs for {count} tensors")
        q = _addresses("grad_clip", out, dev)
        if _sizes_types("grad_clip", out) != (n, t):
            raise FalqError("grad_clip: out must have the tensors' types and sizes")
    norm_at = _arg(norm, torch.float32, (1,), dev, "norm")
    w = _scratch(ws, lib.grad_norm_workspace_bytes(count), dev, stream, st)
    _run(lib.grad_clip, "grad_clip", dev, count, _at(p), _at(n), _at(t), max_norm, eps,
         None if q is None else _at(q), norm_at, *_span(w), st)


# ---------------------------------------------------------------------------
# Microscaled formats (a power of two per block of 32), activations kept in 8 bits,
# and the loss over the vocabulary; as above, on the device of their tensors.

def mxfp4_scales_shape(rows: int, K: int):
    """The shape of the exponent bytes of FP4 operands [rows x K]: steps of 256
    elements, rows up to a multiple of 16, the eight blocks of a step (block b at
    2 (b % 4) + b // 4)."""
    return ((K + 255) // 256, (rows + 15) // 16 * 16, 8)


def mxfp4_scale_bytes(rows: int, K: int) -> int:
    return int(load().mxfp4_scale_bytes(rows, K))


def _mx_operand(q: torch.Tensor, e: torch.Tensor, K: int, dev: int, name: str, ename: str):
    rows = q.shape[0]
    return (_arg(q, torch.uint8, (rows, K // 2), dev, name),
            _arg(e, torch.uint8, mxfp4_scales_shape(rows, K), dev, ename))


def _mx_width(K: int, name: str) -> int:
    if K % 32:
        raise FalqError(f"{name}: rows must be whole blocks of 32, not {K} elements")
    return K


def mxfp4_quantize(x: torch.Tensor, q: torch.Tensor, e: torch.Tensor, stream=None) -> None:
    """FP4 E2M1 codes q [rows x K / 2] (two a byte, the lower index in the low half)
    and exponent bytes e (mxfp4_scales_shape) of x [rows x K], float32 or bfloat16: a
    power of two per block of 32, floor(log2(largest)) - 2; values to nearest, ties to
    the even code, saturating at 6."""
    rows, K = _matrix(x, "x")
    t, dev = _elem(x, "x"), _device(x, "x")
    args = (_arg(x, x.dtype, (rows, _mx_width(K, "x")), dev, "x"), t, rows, K,
            _arg(q, torch.uint8, (rows, K // 2), dev, "q"),
            _arg(e, torch.uint8, mxfp4_scales_shape(rows, K), dev, "e"))
    _run(load().mxfp4_quantize, "mxfp4_quantize", dev, *args, _stream_of(dev, stream))


def mxfp4_dequantize(q: torch.Tensor, e: torch.Tensor, x: torch.Tensor, stream=None) -> None:
    """x [rows x K], float32 or bfloat16, from mxfp4_quantize's codes and exponents."""
    rows, K = _matrix(x, "x")
    t, dev = _elem(x, "x"), _device(q, "q")
    args = (_arg(q, torch.uint8, (rows, _mx_width(K, "x") // 2), dev, "q"),
            _arg(e, torch.uint8, mxfp4_scales_shape(rows, K), dev, "e"), rows, K,
            _arg(x, x.dtype, (rows, K), dev, "x"), t)
    _run(load().mxfp4_dequantize, "mxfp4_dequantize", dev, *args, _stream_of(dev, stream))


def melded_linear_fwd_mxfp4_workspace_bytes(T: int, d_in: int, d_out: int) -> int:
    return int(load().melded_linear_fwd_mxfp4_workspace_bytes(T, d_in, d_out))


def melded_linear_fwd_mxfp4(xq: torch.Tensor, x_e: torch.Tensor, wq: torch.Tensor,
                            w_e: torch.Tensor, y: torch.Tensor,
                            bias: Optional[torch.Tensor] = None, act: str = "none",
                            residual: Optional[torch.Tensor] = None,
                            z: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """melded_linear_fwd_act of mxfp4_quantize's operands: z = dec(xq) dec(wq)^T + bias
    and y = act(z) + residual; xq [T x d_in / 2], wq [d_out x d_in / 2]."""
    T, half = _matrix(xq, "xq")
    d_in, d_out = _mx_width(2 * half, "xq"), _matrix(wq, "wq")[0]
    t, a, dev = _elem(y, "y"), _act(act), _device(xq, "xq")
    f32, out = torch.float32, (T, d_out)
    lib, st = load(), _stream_of(dev, stream)
    args = (*_mx_operand(xq, x_e, d_in, dev, "xq", "x_e"),
            *_mx_operand(wq, w_e, d_in, dev, "wq", "w_e"), _arg(bias, f32, (d_out,), dev, "bias"),
            a, _arg(residual, y.dtype, out, dev, "residual"), T, d_in, d_out, t,
            _arg(y, y.dtype, out, dev, "y"), _arg(z, y.dtype, out, dev, "z"))
    need = 0 if T <= 16 else lib.melded_linear_fwd_mxfp4_workspace_bytes(T, d_in, d_out)
    w = _scratch(ws, need, dev, stream, st)
    _run(lib.melded_linear_fwd_mxfp4, "melded_linear_fwd_mxfp4", dev, *args, *_span(w), st)


def checkpoint_scales_shape(T: int, d: int):
    """The shape of an 8-bit checkpoint's exponent bytes."""
    return (T, (d + 31) // 32)


def _checkpoint(q: torch.Tensor, e: torch.Tensor, T: int, d: int, dev: int, name: str,
                ename: str):
    return (_arg(q, torch.uint8, (T, d), dev, name),
            _arg(e, torch.uint8, checkpoint_scales_shape(T, d), dev, ename))


def checkpoint_save(x: torch.Tensor, q: torch.Tensor, e: torch.Tensor, stream=None) -> None:
    """An activation x [T x d], float32 or bfloat16, kept in 8 bits: E4M3 codes q
    [T x d] and exponent bytes e (checkpoint_scales_shape), a power of two per block of
    32 of a row, the smallest under which the block does not saturate."""
    T, d = _matrix(x, "x")
    t, dev = _elem(x, "x"), _device(x, "x")
    _run(load().checkpoint_save, "checkpoint_save", dev, _arg(x, x.dtype, (T, d), dev, "x"), t, T,
         d, *_checkpoint(q, e, T, d, dev, "q", "e"), _stream_of(dev, stream))


def checkpoint_restore(q: torch.Tensor, e: torch.Tensor, x: torch.Tensor, stream=None) -> None:
    """x [T x d], float32 or bfloat16, from checkpoint_save's codes and exponents."""
    T, d = _matrix(x, "x")
    t, dev = _elem(x, "x"), _device(q, "q")
    _run(load().checkpoint_restore, "checkpoint_restore", dev,
         *_checkpoint(q, e, T, d, dev, "q", "e"), T, d, _arg(x, x.dtype, (T, d), dev, "x"), t,
         _stream_of(dev, stream))


def linear_act_bwd_ckpt(dy: torch.Tensor, z_q: torch.Tensor, z_e: torch.Tensor,
                        dz: Optional[torch.Tensor], dbias: Optional[torch.Tensor] = None,
                        act: str = "none", ws: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """linear_act_bwd with the z of a checkpoint (checkpoint_save's z_q and z_e)."""
    T, d_out = _matrix(dy, "dy")
    gt, a, dev, lib = _elem(dy, "dy"), _act(act), _device(dy, "dy"), load()
    st = _stream_of(dev, stream)
    args = (_arg(dy, dy.dtype, (T, d_out), dev, "dy"), gt,
            *_checkpoint(z_q, z_e, T, d_out, dev, "z_q", "z_e"), a, T, d_out,
            _arg(dz, dy.dtype, (T, d_out), dev, "dz"),
            _arg(dbias, torch.float32, (d_out,), dev, "dbias"))
    need = 0 if dbias is None else lib.linear_act_bwd_workspace_bytes(T, d_out)
    w = _scratch(ws, need, dev, stream, st)
    _run(lib.linear_act_bwd_ckpt, "linear_act_bwd_ckpt", dev, *args, *_span(w), st)


def layer_norm_bwd_ckpt(dy: torch.Tensor, x_q: torch.Tensor, x_e: torch.Tensor,
                        weight: Optional[torch.Tensor], mean: torch.Tensor, rstd: torch.Tensor,
                        dx: Optional[torch.Tensor], dweight: Optional[torch.Tensor] = None,
                        dbias: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """layer_norm_bwd with the x of a checkpoint (checkpoint_save's x_q and x_e); mean
    and rstd are the forward's."""
    T, d = _matrix(dy, "dy")
    gt, dev, f32, lib = _elem(dy, "dy"), _device(dy, "dy"), torch.float32, load()
    st = _stream_of(dev, stream)
    args = (_arg(dy, dy.dtype, (T, d), dev, "dy"), gt,
            *_checkpoint(x_q, x_e, T, d, dev, "x_q", "x_e"), _arg(weight, f32, (d,), dev, "weight"),
            _arg(mean, f32, (T,), dev, "mean"), _arg(rstd, f32, (T,), dev, "rstd"), T, d,
            _arg(dx, dy.dtype, (T, d), dev, "dx"), _arg(dweight, f32, (d,), dev, "dweight"),
            _arg(dbias, f32, (d,), dev, "dbias"))
    need = (0 if dweight is None and dbias is None
            else lib.layer_norm_bwd_workspace_bytes(T, d))
    w = _scratch(ws, need, dev, stream, st)
    _run(lib.layer_norm_bwd_ckpt, "layer_norm_bwd_ckpt", dev, *args, *_span(w), st)


def linear_cross_entropy_fwd_workspace_bytes(T: int, d: int, V: int) -> int:
    return int(load().linear_cross_entropy_fwd_workspace_bytes(T, d, V))


def linear_cross_entropy_fwd(xq: torch.Tensor, s_x: torch.Tensor, wq: torch.Tensor,
                             s_w: torch.Tensor, target: torch.Tensor, loss: torch.Tensor,
                             lse: Optional[torch.Tensor] = None,
                             ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """loss [T] = lse - z[t][target[t]] with the logits z = dec(xq) dec(wq)^T /
    (s_x s_w) over the V rows of wq [V x d], which are not kept, and lse [T] =
    log sum_v exp(z), the backward's input.  target [T] int64; a negative one does
    not count (loss 0)."""
    T, d = _matrix(xq, "xq")
    V, dev = _matrix(wq, "wq")[0], _device(xq, "xq")
    u8, f32, lib, st = torch.uint8, torch.float32, load(), _stream_of(dev, stream)
    args = (_arg(xq, u8, (T, d), dev, "xq"), _arg(s_x, f32, (1,), dev, "s_x"),
            _arg(wq, u8, (V, d), dev, "wq"), _arg(s_w, f32, (1,), dev, "s_w"),
            _arg(target, torch.int64, (T,), dev, "target"), T, d, V,
            _arg(loss, f32, (T,), dev, "loss"), _arg(lse, f32, (T,), dev, "lse"))
    w = _scratch(ws, lib.linear_cross_entropy_fwd_workspace_bytes(T, d, V), dev, stream, st)
    _run(lib.linear_cross_entropy_fwd, "linear_cross_entropy_fwd", dev, *args, *_span(w), st)


def linear_cross_entropy_bwd_workspace_bytes(T: int, d: int, V: int,
                                             dx_dtype=torch.float32) -> int:
    if dx_dtype not in _ELEM:
        raise FalqError(f"dx_dtype: expected float32 or bfloat16, got {dx_dtype}")
    return int(load().linear_cross_entropy_bwd_workspace_bytes(T, d, V, _ELEM[dx_dtype]))


def linear_cross_entropy_bwd(xq: torch.Tensor, s_x: torch.Tensor, wq: torch.Tensor,
                             s_w: torch.Tensor, target: torch.Tensor, lse: torch.Tensor,
                             dloss: torch.Tensor, dx: torch.Tensor,
                             ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """dx [T x d] (float32 or bfloat16), the gradient in x of sum_t dloss[t] loss[t]:
    dloss[t] sum_v (exp(z[t][v] - lse[t]) - [v = target[t]]) dec(wq[v]) / s_w, the
    logits z formed again a piece of the vocabulary at a time.  In float32 to its
    precision; in bfloat16 from FP8's logits and in half the time (falqon.h says how far
    either is off)."""
    T, d = _matrix(xq, "xq")
    V, dev = _matrix(wq, "wq")[0], _device(xq, "xq")
    u8, f32, lib, st = torch.uint8, torch.float32, load(), _stream_of(dev, stream)
    t = _elem(dx, "dx")
    args = (_arg(xq, u8, (T, d), dev, "xq"), _arg(s_x, f32, (1,), dev, "s_x"),
            _arg(wq, u8, (V, d), dev, "wq"), _arg(s_w, f32, (1,), dev, "s_w"),
            _arg(target, torch.int64, (T,), dev, "target"), _arg(lse, f32, (T,), dev, "lse"),
            _arg(dloss, f32, (T,), dev, "dloss"), T, d, V, _arg(dx, dx.dtype, (T, d), dev, "dx"),
            t)
    w = _scratch(ws, lib.linear_cross_entropy_bwd_workspace_bytes(T, d, V, t), dev, stream, st)
    _run(lib.linear_cross_entropy_bwd, "linear_cross_entropy_bwd", dev, *args, *_span(w), st)


from .step import (LinearCrossEntropy, MeldedLinear,  # noqa: E402  (buffers + the call
                   clip_gradients)                    # sequence)
__all__ += ["MeldedLinear", "LinearCrossEntropy", "clip_gradients"]
