"""Python binding of the fp8bs C ABI (include/fp8bs.h).

Fine-grained FP8 quantisation and block-scaled FP8 GEMM on GB300 (sm_103a),
after DeepSeek-V3 "Infrastructure" §3.3.  Every step runs in the CUDA
library ``_build/libfp8bs.so``; this module only marshals arguments
(tensors -> device pointers, the current torch stream) and turns non-zero
status codes into exceptions.  There is no CPU path: if the library is
missing or fails to load, every call raises.

The functions named ``fp8bs_*`` mirror the C entry points one to one and
take tensors or raw device pointers.  ``quantize_act``, ``quantize_weight``,
``gemm`` and ``grouped_gemm`` additionally allocate their outputs with torch,
as the 4-bit and routing functions do.  ``stream`` (a torch stream or a handle)
is the one launched on, torch's current stream by default; outputs belong to
it, and reading them on another one takes the caller's wait, as with any
tensor computed on another stream.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import threading

from .build import LIB_PATH, build as _build

__all__ = [
    "Fp8bsError", "load_library", "build",
    "fp8bs_quantize_act", "fp8bs_quantize_weight", "fp8bs_gemm", "fp8bs_grouped_gemm",
    "fp8bs_gemm_pow2", "fp8bs_grouped_gemm_pow2",
    "fp8bs_gather_q_rows", "fp8bs_scatter_q_rows", "fp8bs_gather_bf16_rows", "fp8bs_moe_combine", "SCALES_KB_MAJOR",
    "SCALES_ROW_MAJOR",
    "fp8bs_quantize_act_ex", "fp8bs_quantize_weight_ex", "fp8bs_quantize_act_weight", "quantize_act_weight", "fp8bs_requant_1x128_to_128x1", "fp8bs_swiglu_quantize",
    "fp8bs_get_device_status", "fp8bs_set_wait_timeout_ms", "fp8bs_status_string", "fp8bs_selftest_wait_timeout",
    "fp8bs_diag_gemm_unpromoted", "diag_gemm_unpromoted",
    "quantize_act", "quantize_weight", "gemm", "grouped_gemm", "requant_1x128_to_128x1", "swiglu_quantize",
    "OUT_F32", "OUT_BF16", "SCALE_BLOCK128x128", "SCALE_ROW1x128", "SCALE_ABSMAX", "SCALE_POW2",
    "fp8bs_fp4_scale_bytes", "fp8bs_quantize_fp4", "fp8bs_swiglu_quantize_fp4", "fp8bs_dequantize_fp4",
    "fp8bs_gemm_fp4", "fp8bs_grouped_gemm_fp4", "fp8bs_moe_route", "fp8bs_moe_route_backward", "fp8bs_moe_layout",
    "fp4_scale_bytes", "quantize_fp4", "swiglu_quantize_fp4", "dequantize_fp4", "gemm_fp4", "grouped_gemm_fp4",
    "moe_route", "moe_route_backward", "moe_layout", "moe_layout_rows", "moe_route_workspace_bytes",
    "moe_layout_workspace_bytes", "FP4_E4M3X16", "FP4_UE8M0X32", "IN_F32", "IN_BF16", "SCORE_SOFTMAX",
    "SCORE_SIGMOID",
]

OUT_F32, OUT_BF16 = 0, 1
SCALES_KB_MAJOR, SCALES_ROW_MAJOR = 0, 1
SCALE_BLOCK128x128, SCALE_ROW1x128 = 0, 1
SCALE_ABSMAX, SCALE_POW2 = 0, 1
FP4_E4M3X16, FP4_UE8M0X32 = 0, 1
IN_F32, IN_BF16 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1

STATUS_NAMES = {0: "FP8BS_OK", 1: "FP8BS_ERR_INVALID_ARG", 2: "FP8BS_ERR_SHAPE", 3: "FP8BS_ERR_ALIGNMENT",
                4: "FP8BS_ERR_UNSUPPORTED_ARCH", 5: "FP8BS_ERR_CUDA", 6: "FP8BS_ERR_TIMEOUT",
                7: "FP8BS_ERR_DEVICE_ARG"}


class Fp8bsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


_lib = None
_lock = threading.Lock()

_c_i64, _c_int, _c_vp, _c_f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float
_SIGNATURES = {
    "fp8bs_quantize_act": [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp],
    "fp8bs_quantize_weight": [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp],
    "fp8bs_quantize_act_ex": [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_vp],
    "fp8bs_quantize_weight_ex": [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_vp],
    "fp8bs_quantize_act_weight": [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64,
                                  _c_vp, _c_vp, _c_int, _c_vp],
    "fp8bs_requant_1x128_to_128x1": [_c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_int, _c_vp],
    "fp8bs_swiglu_quantize": [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_int, _c_vp],
    "fp8bs_gemm": [_c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_vp],
    "fp8bs_grouped_gemm": [_c_vp, _c_vp, _c_i64, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_int, _c_i64, _c_i64,
                           _c_vp],
    "fp8bs_gemm_pow2": [_c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_vp],
    "fp8bs_grouped_gemm_pow2": [_c_vp, _c_vp, _c_i64, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_int, _c_i64, _c_i64,
                                _c_vp],
    "fp8bs_gather_q_rows": [_c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_vp, _c_i64, _c_vp, _c_vp, _c_int, _c_vp],
    "fp8bs_scatter_q_rows": [_c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_vp, _c_int, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp,
                             _c_int, _c_vp],
    "fp8bs_gather_bf16_rows": [_c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp, _c_vp],
    "fp8bs_moe_combine": [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_i64, _c_int, _c_vp, _c_vp],
    "fp8bs_get_device_status": [_c_vp],
    "fp8bs_selftest_wait_timeout": [_c_i64, _c_vp],
    "fp8bs_diag_gemm_unpromoted": [_c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_vp],
    "fp8bs_set_wait_timeout_ms": [_c_i64],
    "fp8bs_status_string": [_c_int],
    "fp8bs_fp4_scale_bytes": [_c_i64, _c_i64, _c_int],
    "fp8bs_quantize_fp4": [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64, _c_int, _c_vp, _c_vp, _c_vp, _c_vp],
    "fp8bs_swiglu_quantize_fp4": [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_vp],
    "fp8bs_dequantize_fp4": [_c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_vp, _c_int, _c_i64, _c_vp],
    "fp8bs_gemm_fp4": [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_int, _c_i64, _c_i64, _c_i64,
                       _c_vp],
    "fp8bs_grouped_gemm_fp4": [_c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_int,
                               _c_i64, _c_i64, _c_vp],
    "fp8bs_moe_route": [_c_vp, _c_int, _c_i64, _c_int, _c_i64, _c_int, _c_vp, _c_vp, _c_vp, _c_i64, _c_int, _c_int,
                        _c_f32, _c_f32, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp],
    "fp8bs_moe_route_workspace_bytes": [_c_i64, _c_int, _c_i64],
    "fp8bs_moe_route_backward": [_c_vp, _c_int, _c_i64, _c_int, _c_i64, _c_int, _c_vp, _c_vp, _c_i64, _c_int, _c_int,
                                 _c_f32, _c_f32, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp],
    "fp8bs_moe_layout": [_c_vp, _c_i64, _c_int, _c_int, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp],
    "fp8bs_moe_layout_rows": [_c_i64, _c_int, _c_int],
    "fp8bs_moe_layout_workspace_bytes": [_c_i64, _c_int, _c_int],
}

# Results other than a status: sizes in bytes or rows (-1: refused), text.
_RESULTS = {"fp8bs_status_string": ctypes.c_char_p, "fp8bs_fp4_scale_bytes": _c_i64,
            "fp8bs_moe_route_workspace_bytes": _c_i64, "fp8bs_moe_layout_rows": _c_i64,
            "fp8bs_moe_layout_workspace_bytes": _c_i64}


def build(force: bool = False) -> str:
    """Compiles the CUDA library in-tree (nvcc, sm_103a) and returns its path."""
    return _build(force=force)


def load_library(path: str | None = None):
    """Loads libfp8bs.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"fp8bs CUDA library not built: {p} is missing (run build())")
            lib = ctypes.CDLL(p, mode=ctypes.RTLD_LOCAL)
            for name, argtypes in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.argtypes = argtypes
                fn.restype = _RESULTS.get(name, ctypes.c_int)
            _lib = lib
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = None   # torch's current stream as a handle, without building a Stream object


def _current_stream() -> int:
    """The current torch stream's handle.  The first call goes through the
    public API, which also initialises CUDA; it takes 2.9 us on the host, more
    than a small kernel's launch, so later ones ask torch for the handle alone
    (0.1 us)."""
    global _raw_stream
    if _raw_stream is not None:
        return _raw_stream[0](_raw_stream[1]())
    import torch
    handle = torch.cuda.current_stream().cuda_stream
    get, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
    if get is not None and device is not None:
        _raw_stream = get, device
    return handle


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != 0:
        raise Fp8bsError(status, where)


# ------------------------------------------------------------ raw C entry points

def fp8bs_quantize_act(x, M, K, ldx, xq, sx, xq_t=None, sx_t=None, stream=None):
    lib = load_library()
    _check(lib.fp8bs_quantize_act(_ptr(x), M, K, ldx, _ptr(xq), _ptr(sx), _ptr(xq_t), _ptr(sx_t),
                                  _stream(stream)), "fp8bs_quantize_act")


def fp8bs_quantize_weight(w, N, K, ldw, wq, sw, wq_t=None, sw_t=None, stream=None):
    lib = load_library()
    _check(lib.fp8bs_quantize_weight(_ptr(w), N, K, ldw, _ptr(wq), _ptr(sw), _ptr(wq_t), _ptr(sw_t),
                                     _stream(stream)), "fp8bs_quantize_weight")


def fp8bs_quantize_act_ex(x, M, K, ldx, xq, sx, xq_t=None, sx_t=None, scale_mode=SCALE_ABSMAX, stream=None):
    lib = load_library()
    _check(lib.fp8bs_quantize_act_ex(_ptr(x), M, K, ldx, _ptr(xq), _ptr(sx), _ptr(xq_t), _ptr(sx_t),
                                     int(scale_mode), _stream(stream)), "fp8bs_quantize_act_ex")


def fp8bs_quantize_weight_ex(w, N, K, ldw, wq, sw, wq_t=None, sw_t=None, scale_mode=SCALE_ABSMAX, stream=None):
    lib = load_library()
    _check(lib.fp8bs_quantize_weight_ex(_ptr(w), N, K, ldw, _ptr(wq), _ptr(sw), _ptr(wq_t), _ptr(sw_t),
                                        int(scale_mode), _stream(stream)), "fp8bs_quantize_weight_ex")


def fp8bs_requant_1x128_to_128x1(xq, sx, M, K, xq_t, sx_t, scale_mode=SCALE_POW2, stream=None):
    lib = load_library()
    _check(lib.fp8bs_requant_1x128_to_128x1(_ptr(xq), _ptr(sx), M, K, _ptr(xq_t), _ptr(sx_t), int(scale_mode),
                                            _stream(stream)), "fp8bs_requant_1x128_to_128x1")


def fp8bs_swiglu_quantize(h, M, I, ldh, q, s, scale_mode=SCALE_ABSMAX, stream=None):
    lib = load_library()
    _check(lib.fp8bs_swiglu_quantize(_ptr(h), M, I, ldh, _ptr(q), _ptr(s), int(scale_mode), _stream(stream)),
           "fp8bs_swiglu_quantize")


def fp8bs_gemm(a, sa, b, sb, sb_kind, d, d_dtype, M, N, K, accumulate=0, stream=None):
    lib = load_library()
    _check(lib.fp8bs_gemm(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), sb_kind, _ptr(d), d_dtype, M, N, K,
                          int(accumulate), _stream(stream)), "fp8bs_gemm")


def fp8bs_grouped_gemm(a, sa, M_total, offsets, num_groups, b, sb, d, d_dtype, N, K, stream=None):
    lib = load_library()
    _check(lib.fp8bs_grouped_gemm(_ptr(a), _ptr(sa), M_total, _ptr(offsets), num_groups, _ptr(b), _ptr(sb),
                                  _ptr(d), d_dtype, N, K, _stream(stream)), "fp8bs_grouped_gemm")


def fp8bs_gemm_pow2(a, sa, b, sb, sb_kind, d, d_dtype, M, N, K, accumulate=0, stream=None):
    lib = load_library()
    _check(lib.fp8bs_gemm_pow2(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), sb_kind, _ptr(d), d_dtype, M, N, K,
                               int(accumulate), _stream(stream)), "fp8bs_gemm_pow2")


def fp8bs_grouped_gemm_pow2(a, sa, M_total, offsets, num_groups, b, sb, d, d_dtype, N, K, stream=None):
    lib = load_library()
    _check(lib.fp8bs_grouped_gemm_pow2(_ptr(a), _ptr(sa), M_total, _ptr(offsets), num_groups, _ptr(b), _ptr(sb),
                                       _ptr(d), d_dtype, N, K, _stream(stream)), "fp8bs_grouped_gemm_pow2")


def fp8bs_gather_q_rows(q, s, rows_in, H, s_in_layout, idx, rows_out, q_out, s_out, s_out_layout, stream=None):
    _check(load_library().fp8bs_gather_q_rows(_ptr(q), _ptr(s), rows_in, H, int(s_in_layout), _ptr(idx), rows_out,
                                              _ptr(q_out), _ptr(s_out), int(s_out_layout), _stream(stream)),
           "fp8bs_gather_q_rows")


def fp8bs_scatter_q_rows(q, s, rows_in, H, s_in_layout, pos, k, zero_rows, n_zero, rows_out, q_out, s_out,
                         s_out_layout, stream=None):
    _check(load_library().fp8bs_scatter_q_rows(_ptr(q), _ptr(s), rows_in, H, int(s_in_layout), _ptr(pos), int(k),
                                               _ptr(zero_rows), n_zero, rows_out, _ptr(q_out), _ptr(s_out),
                                               int(s_out_layout), _stream(stream)),
           "fp8bs_scatter_q_rows")


def fp8bs_gather_bf16_rows(y, rows_in, N, idx, rows_out, out, stream=None):
    _check(load_library().fp8bs_gather_bf16_rows(_ptr(y), rows_in, N, _ptr(idx), rows_out, _ptr(out), _stream(stream)),
           "fp8bs_gather_bf16_rows")


def fp8bs_moe_combine(y, rows_y, N, idx, w, T, k, out, stream=None):
    _check(load_library().fp8bs_moe_combine(_ptr(y), rows_y, N, _ptr(idx), _ptr(w), T, int(k), _ptr(out),
                                            _stream(stream)), "fp8bs_moe_combine")


def fp8bs_get_device_status(stream=None) -> int:
    return load_library().fp8bs_get_device_status(_stream(stream))


def fp8bs_selftest_wait_timeout(timeout_us: int, stream=None):
    _check(load_library().fp8bs_selftest_wait_timeout(int(timeout_us), _stream(stream)), "fp8bs_selftest_wait_timeout")


def fp8bs_quantize_act_weight(x, M, K, ldx, xq, sx, w, N, Kw, ldw, wq, sw, scale_mode=0, stream=None):
    _check(load_library().fp8bs_quantize_act_weight(_ptr(x), M, K, ldx, _ptr(xq), _ptr(sx), _ptr(w), N, Kw, ldw,
                                                    _ptr(wq), _ptr(sw), int(scale_mode), _stream(stream)),
           "fp8bs_quantize_act_weight")


def fp8bs_diag_gemm_unpromoted(a, b, d, M, N, K, stream=None):
    _check(load_library().fp8bs_diag_gemm_unpromoted(_ptr(a), _ptr(b), _ptr(d), M, N, K, _stream(stream)),
           "fp8bs_diag_gemm_unpromoted")


def fp8bs_set_wait_timeout_ms(ms: int):
    _check(load_library().fp8bs_set_wait_timeout_ms(int(ms)), "fp8bs_set_wait_timeout_ms")


def fp8bs_status_string(status: int) -> str:
    return load_library().fp8bs_status_string(int(status)).decode()


def fp8bs_quantize_fp4(x, rows_in, K, ldx, rows, M, fmt, q, sf, g, stream=None):
    _check(load_library().fp8bs_quantize_fp4(_ptr(x), rows_in, K, ldx, _ptr(rows), M, int(fmt), _ptr(q), _ptr(sf),
                                             _ptr(g), _stream(stream)), "fp8bs_quantize_fp4")


def fp8bs_swiglu_quantize_fp4(h, M, I, ldh, live, fmt, q, sf, g, stream=None):
    _check(load_library().fp8bs_swiglu_quantize_fp4(_ptr(h), M, I, ldh, _ptr(live), int(fmt), _ptr(q), _ptr(sf),
                                                    _ptr(g), _stream(stream)), "fp8bs_swiglu_quantize_fp4")


def fp8bs_dequantize_fp4(q, sf, g, M, K, fmt, out, out_dtype, ldo, stream=None):
    _check(load_library().fp8bs_dequantize_fp4(_ptr(q), _ptr(sf), _ptr(g), M, K, int(fmt), _ptr(out), int(out_dtype),
                                               ldo, _stream(stream)), "fp8bs_dequantize_fp4")


def fp8bs_gemm_fp4(a, sfa, ga, b, sfb, gb, fmt, d, d_dtype, M, N, K, stream=None):
    _check(load_library().fp8bs_gemm_fp4(_ptr(a), _ptr(sfa), _ptr(ga), _ptr(b), _ptr(sfb), _ptr(gb), int(fmt), _ptr(d),
                                         int(d_dtype), M, N, K, _stream(stream)), "fp8bs_gemm_fp4")


def fp8bs_grouped_gemm_fp4(a, sfa, ga, M_total, offsets, num_groups, b, sfb, gb, fmt, d, d_dtype, N, K, stream=None):
    _check(load_library().fp8bs_grouped_gemm_fp4(_ptr(a), _ptr(sfa), _ptr(ga), M_total, _ptr(offsets), num_groups,
                                                 _ptr(b), _ptr(sfb), _ptr(gb), int(fmt), _ptr(d), int(d_dtype), N, K,
                                                 _stream(stream)), "fp8bs_grouped_gemm_fp4")


def fp8bs_moe_route(logits, in_dtype, T, E, ld, score, bias, valid, seq, S, k, normalize, scale, alpha, idx, w, counts,
                    tokens, loss, ws, ws_bytes, stream=None):
    _check(load_library().fp8bs_moe_route(_ptr(logits), int(in_dtype), T, E, ld, int(score), _ptr(bias), _ptr(valid),
                                          _ptr(seq), S, k, int(normalize), scale, alpha, _ptr(idx), _ptr(w),
                                          _ptr(counts), _ptr(tokens), _ptr(loss), _ptr(ws), ws_bytes,
                                          _stream(stream)), "fp8bs_moe_route")


def fp8bs_moe_route_backward(logits, in_dtype, T, E, ld, score, valid, seq, S, k, normalize, scale, alpha, idx, counts,
                             tokens, dw, dloss, dlogits, ldd, stream=None):
    _check(load_library().fp8bs_moe_route_backward(_ptr(logits), int(in_dtype), T, E, ld, int(score), _ptr(valid),
                                                   _ptr(seq), S, k, int(normalize), scale, alpha, _ptr(idx),
                                                   _ptr(counts), _ptr(tokens), _ptr(dw), _ptr(dloss), _ptr(dlogits),
                                                   ldd, _stream(stream)), "fp8bs_moe_route_backward")


def fp8bs_moe_layout(idx, T, k, E, offsets, row_token, rows, row_of, ws, ws_bytes, stream=None):
    _check(load_library().fp8bs_moe_layout(_ptr(idx), T, k, E, _ptr(offsets), _ptr(row_token), rows, _ptr(row_of),
                                           _ptr(ws), ws_bytes, _stream(stream)), "fp8bs_moe_layout")


def _size(name: str, *args) -> int:
    n = getattr(load_library(), name)(*args)
    if n < 0:
        raise Fp8bsError(1, name)
    return n


def fp8bs_fp4_scale_bytes(M: int, K: int, fmt: int) -> int:
    return _size("fp8bs_fp4_scale_bytes", M, K, int(fmt))


def moe_route_workspace_bytes(T: int, E: int, S: int = 1) -> int:
    return _size("fp8bs_moe_route_workspace_bytes", T, E, S)


def moe_layout_rows(T: int, k: int, E: int) -> int:
    """The most rows that the padded segments of T tokens' k choices among E experts can take."""
    return _size("fp8bs_moe_layout_rows", T, k, E)


def moe_layout_workspace_bytes(T: int, k: int, E: int) -> int:
    return _size("fp8bs_moe_layout_workspace_bytes", T, k, E)


fp4_scale_bytes = fp8bs_fp4_scale_bytes


# ------------------------------------------------------ allocating conveniences

def _allocates_on_its_stream(fn):
    """For a function that allocates tensors and launches on ``stream``: where
    that is not torch's current stream, the tensors are allocated for it.  A
    block that the current stream freed may still be written by work queued
    there, which orders nothing on another stream; and scratch freed on return
    goes back to the stream that still uses it.  The outputs are then marked as
    used on the current stream too, where the caller most likely reads them, so
    that the allocator keeps them for what is queued there when they are freed."""
    place = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kwargs):
        stream = args[place] if len(args) > place else kwargs.get("stream")
        if stream is None:
            return fn(*args, **kwargs)
        import torch
        current, handle = torch.cuda.current_stream(), _stream(stream)
        if handle == current.cuda_stream:
            return fn(*args, **kwargs)
        with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(handle)):
            out = fn(*args, **kwargs)
        for t in out if isinstance(out, tuple) else (out,):
            if t is not None:
                t.record_stream(current)
        return out

    return call


def _checked(t, name: str, dtypes, dim: int | None = None, rows: bool = False):
    """A tensor of one of the given types (and number of dimensions), its last
    dimension dense; all of it dense unless ``rows``.  The C entry points see
    pointers only."""
    if not t.is_cuda:
        raise ValueError(f"{name}: not a CUDA tensor")
    if t.dtype not in dtypes or (dim is not None and t.dim() != dim):
        raise ValueError(f"{name}: {t.dim()}-d {t.dtype}; expected {dim}-d {' or '.join(map(str, dtypes))}")
    if (t.stride(-1) != 1 and t.shape[-1] > 1) if rows else not t.is_contiguous():
        raise ValueError(f"{name}: strides {tuple(t.stride())} of shape {tuple(t.shape)}")
    return t


def _out_type(dtype):
    """(torch type, fp8bs_out_dtype) of an output: bfloat16 (default) or float32.
    The kernels write two or four bytes an element, so any other type is
    refused before it is allocated."""
    import torch
    dtype = dtype or torch.bfloat16
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"out_dtype: {dtype}; expected torch.bfloat16 or torch.float32")
    return dtype, OUT_BF16 if dtype == torch.bfloat16 else OUT_F32


def _product_out(out, out_dtype, M, N, device):
    """(output [M, N], its fp8bs_out_dtype): the given one, checked, or a new one."""
    import torch
    if out is None:
        dtype, code = _out_type(out_dtype)
        return torch.empty((M, N), dtype=dtype, device=device), code
    if tuple(_checked(out, "out", (torch.bfloat16, torch.float32), 2).shape) != (M, N):
        raise ValueError(f"out: shape {tuple(out.shape)}, expected {(M, N)}")
    return out, _out_type(out.dtype)[1]


@_allocates_on_its_stream
def quantize_act(x, transposed: bool = False, pow2: bool = False, stream=None):
    """x: [M, K] bfloat16 CUDA tensor (row-major, K % 128 == 0).

    Returns (xq [M,K] uint8, sx [K/128, M] float32) and, with ``transposed``,
    also (xq_t [K,M] uint8, sx_t [M/128, K] float32).  ``pow2`` selects
    power-of-two scales (SCALE_POW2).
    """
    import torch
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    sx = torch.empty((K // 128, M), dtype=torch.float32, device=x.device)
    xq_t = sx_t = None
    if transposed:
        xq_t = torch.empty((K, M), dtype=torch.uint8, device=x.device)
        sx_t = torch.empty((M // 128, K), dtype=torch.float32, device=x.device)
    fp8bs_quantize_act_ex(x, M, K, x.stride(0), xq, sx, xq_t, sx_t, SCALE_POW2 if pow2 else SCALE_ABSMAX, stream)
    return (xq, sx, xq_t, sx_t) if transposed else (xq, sx)


@_allocates_on_its_stream
def quantize_weight(w, transposed: bool = False, pow2: bool = False, stream=None):
    """w: [N, K] bfloat16 CUDA tensor.  Returns (wq, sw[, wq_t, sw_t])."""
    import torch
    N, K = w.shape
    wq = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    sw = torch.empty((N // 128, K // 128), dtype=torch.float32, device=w.device)
    wq_t = sw_t = None
    if transposed:
        wq_t = torch.empty((K, N), dtype=torch.uint8, device=w.device)
        sw_t = torch.empty((K // 128, N // 128), dtype=torch.float32, device=w.device)
    fp8bs_quantize_weight_ex(w, N, K, w.stride(0), wq, sw, wq_t, sw_t, SCALE_POW2 if pow2 else SCALE_ABSMAX, stream)
    return (wq, sw, wq_t, sw_t) if transposed else (wq, sw)


@_allocates_on_its_stream
def swiglu_quantize(h, pow2: bool = False, stream=None):
    """h: [M, 2I] bfloat16 CUDA tensor (gate | up).  Returns (q [M, I] uint8,
    s [I/128, M] float32): the 1x128 quantisation of BF16(silu(gate) * up)."""
    import torch
    M, two_i = h.shape
    I = two_i // 2
    q = torch.empty((M, I), dtype=torch.uint8, device=h.device)
    s = torch.empty((I // 128, M), dtype=torch.float32, device=h.device)
    fp8bs_swiglu_quantize(h, M, I, h.stride(0), q, s, SCALE_POW2 if pow2 else SCALE_ABSMAX, stream)
    return q, s


@_allocates_on_its_stream
def requant_1x128_to_128x1(xq, sx, pow2: bool = True, stream=None):
    """Re-tile 1x128-quantised activations (xq [M,K] uint8, sx [K/128, M]) into
    128x1 groups: returns (xq_t [K,M] uint8, sx_t [M/128, K] float32)."""
    import torch
    M, K = xq.shape
    xq_t = torch.empty((K, M), dtype=torch.uint8, device=xq.device)
    sx_t = torch.empty((M // 128, K), dtype=torch.float32, device=xq.device)
    fp8bs_requant_1x128_to_128x1(xq, sx, M, K, xq_t, sx_t, SCALE_POW2 if pow2 else SCALE_ABSMAX, stream)
    return xq_t, sx_t


@_allocates_on_its_stream
def gemm(a, sa, b, sb, sb_kind: int = SCALE_BLOCK128x128, out_dtype=None, out=None, accumulate: bool = False,
         stream=None, pow2: bool = False):
    """D = A B^T with per-128-K-block scales; A [M,K], B [N,K] uint8 E4M3.
    ``pow2``: power-of-two scales applied by the tensor core (fp8bs_gemm_pow2)."""
    M, K = a.shape
    N = b.shape[0]
    out, d_dtype = _product_out(out, out_dtype, M, N, a.device)
    fn = fp8bs_gemm_pow2 if pow2 else fp8bs_gemm
    fn(a, sa, b, sb, sb_kind, out, d_dtype, M, N, K, int(accumulate), stream)
    return out


@_allocates_on_its_stream
def grouped_gemm(a, sa, offsets, b, sb, out_dtype=None, out=None, stream=None, pow2: bool = False):
    """Per-expert D rows = A rows of the expert x B[g]^T; offsets: int32 CUDA tensor [G+1].
    ``pow2``: power-of-two scales applied by the tensor core (fp8bs_grouped_gemm_pow2)."""
    M, K = a.shape
    G, N, _ = b.shape
    out, d_dtype = _product_out(out, out_dtype, M, N, a.device)
    fn = fp8bs_grouped_gemm_pow2 if pow2 else fp8bs_grouped_gemm
    fn(a, sa, M, offsets, G, b, sb, out, d_dtype, N, K, stream)
    return out


@_allocates_on_its_stream
def diag_gemm_unpromoted(a, b, stream=None):
    """Diagnostic: FP32 D = A B^T of E4M3 codes (A [M,K], B [N,K] uint8) with all
    of K accumulated by the tensor core alone, no promotion and no scales."""
    import torch
    M, K = a.shape
    N = b.shape[0]
    out = torch.empty((M, N), dtype=torch.float32, device=a.device)
    fp8bs_diag_gemm_unpromoted(a, b, out, M, N, K, stream)
    return out


@_allocates_on_its_stream
def quantize_act_weight(x, w, pow2: bool = False, stream=None):
    """X [M,K] and W [N,Kw] bfloat16 CUDA tensors quantised in one launch:
    returns (xq, sx [K/128, M], wq, sw [N/128, Kw/128])."""
    import torch
    M, K = x.shape
    N, Kw = w.shape
    xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    sx = torch.empty((K // 128, M), dtype=torch.float32, device=x.device)
    wq = torch.empty((N, Kw), dtype=torch.uint8, device=w.device)
    sw = torch.empty((N // 128, Kw // 128), dtype=torch.float32, device=w.device)
    fp8bs_quantize_act_weight(x, M, K, x.stride(0), xq, sx, w, N, Kw, w.stride(0), wq, sw,
                              SCALE_POW2 if pow2 else SCALE_ABSMAX, stream)
    return xq, sx, wq, sw


def _row_stride(t) -> int:
    return t.stride(-2) if t.shape[-2] > 1 else t.shape[-1]


def _fp4_outputs(lead, K, fmt, device):
    import torch
    q = torch.empty((*lead, K // 2), dtype=torch.uint8, device=device)
    sf = torch.empty((*lead[:-1], fp8bs_fp4_scale_bytes(lead[-1], K, fmt)), dtype=torch.uint8, device=device)
    g = torch.empty(lead, dtype=torch.float32, device=device) if fmt == FP4_E4M3X16 else None
    return q, sf, g


@_allocates_on_its_stream
def quantize_fp4(x, fmt: int = FP4_E4M3X16, rows=None, stream=None):
    """x: [M, K] bfloat16 CUDA tensor (K % 64 == 0), or expert weights [G, N, K]
    (contiguous).  Returns (q [..., K/2] uint8, two E2M1 codes a byte; sf uint8,
    the scales in 512-byte blocks of 128 rows; g float32, a scale per row, None
    for FP4_UE8M0X32).  ``rows``: int32 [M'], quantise x[rows[i]] as row i (a
    row of zeros where rows[i] < 0); x is a matrix then."""
    import torch
    K = x.shape[-1]
    if x.dim() == 3:
        if rows is not None:
            raise ValueError("rows: picks rows of a matrix [M, K], not of expert weights")
        _checked(x, "x", (torch.bfloat16,), 3)
        G, N, _ = x.shape
        q, sf, g = _fp4_outputs((G, N), K, fmt, x.device)
        if N % 128 == 0:      # the experts' scale blocks follow one another
            fp8bs_quantize_fp4(x, G * N, K, K, None, G * N, fmt, q, sf, g, stream)
        else:
            for i in range(G):
                fp8bs_quantize_fp4(x[i], N, K, K, None, N, fmt, q[i], sf[i], None if g is None else g[i], stream)
        return q, sf, g
    _checked(x, "x", (torch.bfloat16,), 2, rows=True)
    if rows is not None:
        _checked(rows, "rows", (torch.int32,), 1)
    M = x.shape[0] if rows is None else rows.shape[0]
    q, sf, g = _fp4_outputs((M,), K, fmt, x.device)
    fp8bs_quantize_fp4(x, x.shape[0], K, _row_stride(x), rows, M, fmt, q, sf, g, stream)
    return q, sf, g


@_allocates_on_its_stream
def swiglu_quantize_fp4(h, fmt: int = FP4_E4M3X16, live=None, stream=None):
    """h: [M, 2I] bfloat16 CUDA tensor (gate | up).  Returns the 4-bit codes and
    scales of BF16(silu(gate) * up), as quantize_fp4; rows with live[i] < 0
    (int32 [M]) are rows of zeros."""
    import torch
    _checked(h, "h", (torch.bfloat16,), 2, rows=True)
    M, two_i = h.shape
    if two_i % 2 != 0:
        raise ValueError(f"h: {two_i} columns; expected as many of the gate as of up")
    if live is not None and _checked(live, "live", (torch.int32,), 1).shape[0] != M:
        raise ValueError("live: one value per row of h")
    q, sf, g = _fp4_outputs((M,), two_i // 2, fmt, h.device)
    fp8bs_swiglu_quantize_fp4(h, M, two_i // 2, _row_stride(h), live, fmt, q, sf, g, stream)
    return q, sf, g


@_allocates_on_its_stream
def dequantize_fp4(q, sf, g=None, fmt: int = FP4_E4M3X16, out_dtype=None, stream=None):
    """The values [M, K] of 4-bit codes, bfloat16 (default) or float32."""
    import torch
    _fp4_operand((q, sf, g), "codes", fmt, 2)
    M, K = q.shape[0], 2 * q.shape[1]
    out_dtype, code = _out_type(out_dtype)
    out = torch.empty((M, K), dtype=out_dtype, device=q.device)
    fp8bs_dequantize_fp4(q, sf, g, M, K, fmt, out, code, K, stream)
    return out


def _fp4_operand(t, name: str, fmt: int, dim: int):
    """Codes, scales and row scales that fit one another."""
    import torch
    q, sf, g = t
    _checked(q, name + " codes", (torch.uint8,), dim)
    _checked(sf, name + " scales", (torch.uint8,))
    need = fp8bs_fp4_scale_bytes(q.shape[-2], 2 * q.shape[-1], fmt) * (q.shape[0] if dim == 3 else 1)
    if sf.numel() != need or (fmt == FP4_E4M3X16 and (g is None or _checked(g, name + " row scales", (torch.float32,)).shape
                                                      != q.shape[:-1])):
        raise ValueError(f"{name}: scales do not fit codes of shape {tuple(q.shape)}")
    return q, sf, g


@_allocates_on_its_stream
def gemm_fp4(a, b, fmt: int = FP4_E4M3X16, out_dtype=None, out=None, stream=None):
    """D = A B^T of 4-bit operands; a = (q [M, K/2], sf, g) and b = (q [N, K/2], sf, g) as
    quantize_fp4 returns them."""
    (qa, sfa, ga), (qb, sfb, gb) = _fp4_operand(a, "a", fmt, 2), _fp4_operand(b, "b", fmt, 2)
    M, N, K = qa.shape[0], qb.shape[0], 2 * qa.shape[1]
    if qb.shape[1] != qa.shape[1]:
        raise ValueError(f"K differs: {K} and {2 * qb.shape[1]}")
    out, d_dtype = _product_out(out, out_dtype, M, N, qa.device)
    fp8bs_gemm_fp4(qa, sfa, ga, qb, sfb, gb, fmt, out, d_dtype, M, N, K, stream)
    return out


@_allocates_on_its_stream
def grouped_gemm_fp4(a, offsets, b, fmt: int = FP4_E4M3X16, out_dtype=None, out=None, stream=None):
    """Per-expert D rows = A rows of the expert x B[g]^T; offsets int32 CUDA tensor [G+1], b as
    quantize_fp4 returns it for weights [G, N, K]."""
    import torch
    (qa, sfa, ga), (qb, sfb, gb) = _fp4_operand(a, "a", fmt, 2), _fp4_operand(b, "b", fmt, 3)
    M, K = qa.shape[0], 2 * qa.shape[1]
    G, N, _ = qb.shape
    if qb.shape[2] != qa.shape[1] or _checked(offsets, "offsets", (torch.int32,), 1).shape[0] != G + 1:
        raise ValueError(f"a {tuple(qa.shape)}, b {tuple(qb.shape)} and {offsets.shape[0]} offsets do not fit")
    out, d_dtype = _product_out(out, out_dtype, M, N, qa.device)
    fp8bs_grouped_gemm_fp4(qa, sfa, ga, M, offsets, G, qb, sfb, gb, fmt, out, d_dtype, N, K, stream)
    return out


def _route_inputs(logits, bias, valid, seq):
    import torch
    _checked(logits, "logits", (torch.float32, torch.bfloat16), 2, rows=True)
    T, E = logits.shape
    if bias is not None and _checked(bias, "bias", (torch.float32,), 1).shape[0] != E:
        raise ValueError("bias: one value per expert")
    if valid is not None and _checked(valid, "valid", (torch.uint8, torch.bool), 1).shape[0] != T:
        raise ValueError("valid: one value per token")
    if seq is not None:
        _checked(seq, "seq", (torch.int32,), 1)


@_allocates_on_its_stream
def moe_route(logits, k: int, score: int = SCORE_SOFTMAX, bias=None, valid=None, seq=None, normalize: bool = True,
              scale: float = 1.0, alpha: float | None = None, stream=None):
    """Expert choice of each token: logits [T, E] float32 or bfloat16.  Returns
    (idx [T, k] int32, w [T, k] float32), and with ``alpha`` (the balance
    loss's factor) also (counts [S, E] int32, tokens [S] int32, loss [1]).
    ``valid``: uint8 [T]; ``seq``: int32 [S + 1], the sequences' first tokens."""
    import torch
    S = 1 if seq is None else seq.shape[0] - 1
    _route_inputs(logits, bias, valid, seq)
    T, E = logits.shape
    dev = logits.device
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    in_dtype = IN_BF16 if logits.dtype == torch.bfloat16 else IN_F32
    ld = _row_stride(logits)
    if alpha is None:
        fp8bs_moe_route(logits, in_dtype, T, E, ld, score, bias, valid, None, 1, k, normalize, scale, 0.0,
                        idx, w, None, None, None, None, 0, stream)
        return idx, w
    counts = torch.empty((S, E), dtype=torch.int32, device=dev)
    tokens = torch.empty(S, dtype=torch.int32, device=dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    n = moe_route_workspace_bytes(T, E, S)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    fp8bs_moe_route(logits, in_dtype, T, E, ld, score, bias, valid, seq, S, k, normalize, scale, alpha, idx, w, counts,
                    tokens, loss, ws, n, stream)
    return idx, w, counts, tokens, loss


@_allocates_on_its_stream
def moe_route_backward(logits, idx, dw, score: int = SCORE_SOFTMAX, valid=None, seq=None, normalize: bool = True,
                       scale: float = 1.0, alpha: float = 0.0, counts=None, tokens=None, dloss=None, stream=None):
    """Gradient of moe_route's weights (dw [T, k]) and balance loss (dloss, one
    float32, with moe_route's counts [S, E] and tokens [S]; None leaves the
    loss out) with respect to the logits, in their type."""
    import torch
    _route_inputs(logits, None, valid, seq)
    T, E = logits.shape
    S = 1 if seq is None else seq.shape[0] - 1
    if _checked(idx, "idx", (torch.int32,), 2).shape != _checked(dw, "dw", (torch.float32,), 2).shape or idx.shape[0] != T:
        raise ValueError(f"idx {tuple(idx.shape)} and dw {tuple(dw.shape)}: one row per token each")
    if dloss is not None:
        if _checked(dloss, "dloss", (torch.float32,)).numel() != 1:
            raise ValueError(f"dloss: {dloss.numel()} values; expected one")
        if counts is None or tokens is None:
            raise ValueError("dloss: needs moe_route's counts and tokens")
        if (tuple(_checked(counts, "counts", (torch.int32,), 2).shape) != (S, E)
                or tuple(_checked(tokens, "tokens", (torch.int32,), 1).shape) != (S,)):
            raise ValueError(f"counts {tuple(counts.shape)} and tokens {tuple(tokens.shape)}: expected {(S, E)} and {(S,)}")
    dlogits = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    fp8bs_moe_route_backward(logits, IN_BF16 if logits.dtype == torch.bfloat16 else IN_F32, T, E, _row_stride(logits),
                             score, valid, seq, S, idx.shape[1], normalize, scale, alpha, idx, counts, tokens, dw,
                             dloss, dlogits, E, stream)
    return dlogits


@_allocates_on_its_stream
def moe_layout(idx, E: int, stream=None):
    """Row layout of the choices idx [T, k] among E experts: (offsets [E + 1], row_token
    [rows], row_of [T, k]), int32, as fp8bs_moe_layout describes them."""
    import torch
    T, k = _checked(idx, "idx", (torch.int32,), 2).shape
    rows = moe_layout_rows(T, k, E)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=idx.device)
    row_token = torch.empty(rows, dtype=torch.int32, device=idx.device)
    row_of = torch.empty((T, k), dtype=torch.int32, device=idx.device)
    n = moe_layout_workspace_bytes(T, k, E)
    ws = torch.empty(n, dtype=torch.uint8, device=idx.device)
    fp8bs_moe_layout(idx, T, k, E, offsets, row_token, rows, row_of, ws, n, stream)
    return offsets, row_token, row_of
