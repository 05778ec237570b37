"""ctypes binding of librazer.so (declared in include/razer.h).

Argument marshalling only: every step of the RaZeR path runs in the CUDA
kernels of the library.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the library is missing or a call fails,
an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librazer.so")

# enums of include/razer.h
RAZER_OK = 0
STATUS_NAMES = {
    0: "RAZER_OK", 1: "RAZER_ERR_INVALID_ARG", 2: "RAZER_ERR_SHAPE", 3: "RAZER_ERR_ALIGN",
    4: "RAZER_ERR_DTYPE", 5: "RAZER_ERR_WORKSPACE", 6: "RAZER_ERR_UNSUPPORTED",
    7: "RAZER_ERR_TIMEOUT", 8: "RAZER_ERR_CUDA",
}
RAZER_F16, RAZER_BF16, RAZER_F32 = 0, 1, 2
RAZER_FMT_WEIGHT, RAZER_FMT_ACT, RAZER_FMT_NVFP4, RAZER_FMT_FOUR_OVER_SIX, RAZER_SCALE_F16, RAZER_FMT_MXFP4 = 0, 1, 2, 3, 4, 5
RAZER_OP_GEMV, RAZER_OP_GEMM, RAZER_OP_GEMM_W4A4, RAZER_OP_GEMM_VARIANT, RAZER_OP_GEMM_MX_ONLINE = 0, 1, 2, 3, 4
RAZER_ACT_NONE, RAZER_ACT_SILU_MUL = 0, 1
ACTS = {None: RAZER_ACT_NONE, "silu_mul": RAZER_ACT_SILU_MUL}
FORMATS = {"weight": RAZER_FMT_WEIGHT, "act": RAZER_FMT_ACT, "nvfp4": RAZER_FMT_NVFP4, "four_over_six": RAZER_FMT_FOUR_OVER_SIX,
           "f16_scale": RAZER_SCALE_F16, "mxfp4": RAZER_FMT_MXFP4}
_DT = {torch.float16: RAZER_F16, torch.bfloat16: RAZER_BF16, torch.float32: RAZER_F32}

EXPORTED = (
    "razer_quantize_weights", "razer_quantize_weights_batch", "razer_quantize_acts", "razer_dequant", "razer_gemv", "razer_gemm",
    "razer_gemv_batch", "razer_gemv_batch_workspace_size", "razer_gemm_w4a4", "razer_gemm_w4a4_online", "razer_quant_error",
    "razer_quantize_variant", "razer_quant_error_variant", "razer_dequant_variant", "razer_gemv_variant", "razer_gemm_variant",
    "razer_workspace_size", "razer_get_device_status", "razer_status_string", "razer_version",
    "razer_gemv_noalloc", "razer_gemv_noalloc_max_scratch", "razer_debug_set_fault_injection", "razer_set_quantize_path",
    "razer_scale_tiles_size", "razer_quantize_mx", "razer_dequant_mx", "razer_tile_scales", "razer_gemm_mx", "razer_gemm_mx_grouped",
    "razer_gemm_mx_online", "razer_gemm_mx_grouped_online", "razer_gemm_mx_grouped_workspace_size",
)


class GemvProblem(ctypes.Structure):
    """razer_gemv_problem of include/razer.h."""
    _fields_ = [("x", ctypes.c_void_p), ("B", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("ts", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("y", ctypes.c_void_p)]


class RazerError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")


_lib = None


def load() -> ctypes.CDLL:
    """Load librazer.so (built in-tree by bit_quantization_razer_b200.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: run `python -m bit_quantization_razer_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    L.razer_quantize_weights.argtypes = [vp, i32, i64, i64, vp, vp, vp, i32, vp]
    L.razer_quantize_weights_batch.argtypes = [i32, ctypes.POINTER(vp), i32, ctypes.POINTER(i64), ctypes.POINTER(i64),
                                               ctypes.POINTER(vp), ctypes.POINTER(vp), vp, i32, vp]
    L.razer_quantize_acts.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp, vp, i32, vp]
    L.razer_dequant.argtypes = [vp, vp, vp, i32, i64, i64, vp, i32, vp]
    L.razer_gemv.argtypes = [vp, i32, i64, vp, vp, vp, i32, i64, i64, vp, i32, vp, sz, vp]
    L.razer_gemm.argtypes = [vp, i32, i64, vp, vp, vp, i32, i64, i64, vp, i32, vp, sz, vp]
    L.razer_gemv_batch.argtypes = [i32, ctypes.POINTER(GemvProblem), i32, i32, i32, vp, sz, vp]
    L.razer_gemm_w4a4.argtypes = [vp, vp, vp, i32, i64, vp, vp, vp, i32, i64, i64, vp, i32, vp, sz, vp]
    L.razer_gemm_w4a4_online.argtypes = [vp, i32, i64, vp, i32, vp, vp, vp, vp, vp, vp, vp, i32, i64, i64, vp, i32, vp, sz, vp]
    L.razer_quantize_variant.argtypes = [vp, i32, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_float), i32, vp, vp, vp, vp]
    L.razer_quant_error_variant.argtypes = [vp, i32, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_float), i32, vp, vp, vp, vp, vp]
    L.razer_dequant_variant.argtypes = [vp, vp, vp, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_float), i32, vp, i32, vp]
    L.razer_gemv_variant.argtypes = [vp, i32, i64, vp, vp, vp, i32, i32, ctypes.POINTER(ctypes.c_float), i32, i64, i64, vp, i32, vp,
                                     sz, vp]
    L.razer_gemm_variant.argtypes = [vp, i32, i64, vp, vp, vp, i32, i32, ctypes.POINTER(ctypes.c_float), i32, i64, i64, vp, i32, vp,
                                     sz, vp]
    L.razer_quant_error.argtypes = [vp, i32, i64, i64, vp, vp, vp, i32, vp, vp]
    L.razer_gemv_batch_workspace_size.argtypes = [i32, ctypes.POINTER(GemvProblem)]
    L.razer_gemv_batch_workspace_size.restype = sz
    L.razer_gemv_noalloc.argtypes = [vp, i32, i64, vp, vp, vp, i32, i64, i64, vp, i32, vp]
    L.razer_gemv_noalloc.restype = ctypes.c_int
    L.razer_gemv_noalloc_max_scratch.argtypes = []
    L.razer_gemv_noalloc_max_scratch.restype = sz
    L.razer_workspace_size.argtypes = [i32, i64, i64, i64]
    L.razer_workspace_size.restype = sz
    L.razer_get_device_status.argtypes = [vp]
    L.razer_status_string.argtypes = [i32]
    L.razer_status_string.restype = ctypes.c_char_p
    L.razer_version.argtypes = []
    L.razer_debug_set_fault_injection.argtypes = [i32]
    L.razer_debug_set_fault_injection.restype = ctypes.c_int
    L.razer_set_quantize_path.argtypes = [i32]
    L.razer_set_quantize_path.restype = ctypes.c_int
    L.razer_scale_tiles_size.argtypes = [i32, i64, i64, i64]
    L.razer_scale_tiles_size.restype = sz
    L.razer_quantize_mx.argtypes = [vp, i32, i64, i64, vp, i64, vp, vp, vp]
    L.razer_dequant_mx.argtypes = [vp, vp, i64, i64, vp, i64, vp, i32, vp]
    L.razer_tile_scales.argtypes = [vp, i64, i64, i64, vp, i64, vp, vp]
    L.razer_gemm_mx.argtypes = [vp, vp, vp, i64, vp, vp, vp, i32, i64, i64, i32, vp, i32, vp]
    L.razer_gemm_mx_grouped.argtypes = [vp, vp, vp, i64, vp, i64, vp, vp, vp, i32, i64, i64, i32, vp, i32, vp]
    L.razer_gemm_mx_online.argtypes = [vp, i32, i64, vp, vp, i64, i64, i32, vp, i32, vp, sz, vp]
    L.razer_gemm_mx_grouped_online.argtypes = [vp, i32, i64, vp, i64, vp, vp, i64, i64, i32, vp, i32, vp, sz, vp]
    L.razer_gemm_mx_grouped_workspace_size.argtypes = [i64, i64, i64]
    L.razer_gemm_mx_grouped_workspace_size.restype = sz
    for fn in ("razer_quantize_mx", "razer_dequant_mx", "razer_tile_scales", "razer_gemm_mx", "razer_gemm_mx_grouped",
               "razer_gemm_mx_online", "razer_gemm_mx_grouped_online", "razer_quantize_variant", "razer_quant_error_variant", "razer_dequant_variant", "razer_gemv_variant", "razer_gemm_variant",
               "razer_gemm_w4a4_online", "razer_quant_error", "razer_gemm_w4a4", "razer_gemv_batch", "razer_quantize_weights", "razer_quantize_weights_batch", "razer_quantize_acts", "razer_dequant", "razer_gemv", "razer_gemm",
               "razer_get_device_status", "razer_version"):
        getattr(L, fn).restype = ctypes.c_int
    _lib = L
    return L


def _p(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, status: int):
    if status != RAZER_OK:
        raise RazerError(fn, status)


def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def razer_quantize_weights(W: torch.Tensor, fmt="weight", *, codes=None, scales=None, ts=None, stream=None):
    """Quantize W [N, K] (fp16/bf16, CUDA). Returns (codes [N, K/2] u8,
    scales [N, K/16] u8, ts [1] f32), all on W's device."""
    N, K = W.shape
    dev = W.device
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev) if codes is None else codes
    scales = torch.empty((N, K // 16), dtype=torch.uint8, device=dev) if scales is None else scales
    ts = torch.empty(1, dtype=torch.float32, device=dev) if ts is None else ts
    st = load().razer_quantize_weights(_p(W), _DT.get(W.dtype, -1), N, K, _p(codes), _p(scales), _p(ts), _fmt(fmt), _stream(stream))
    _check("razer_quantize_weights", st)
    return codes, scales, ts


def razer_quantize_weights_batch(Ws, fmt="weight", *, codes=None, scales=None, ts=None, stream=None):
    """Quantize several weight matrices (same dtype and device) in one call.
    Returns (list of codes, list of scales, ts [count] f32); matrix i's
    results equal razer_quantize_weights(Ws[i])."""
    n = len(Ws)
    dev = Ws[0].device if n else torch.device("cuda")
    dt = _DT.get(Ws[0].dtype, -1) if n else 0
    codes = [torch.empty((w.shape[0], w.shape[1] // 2), dtype=torch.uint8, device=dev) for w in Ws] if codes is None else codes
    scales = [torch.empty((w.shape[0], w.shape[1] // 16), dtype=torch.uint8, device=dev) for w in Ws] if scales is None else scales
    ts = torch.empty(max(n, 1), dtype=torch.float32, device=dev) if ts is None else ts
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    arr = lambda ts_: (vp * max(n, 1))(*[t.data_ptr() for t in ts_])
    Ns = (i64 * max(n, 1))(*[w.shape[0] for w in Ws])
    Ks = (i64 * max(n, 1))(*[w.shape[1] for w in Ws])
    st = load().razer_quantize_weights_batch(n, arr(Ws), dt, Ns, Ks, arr(codes), arr(scales), _p(ts), _fmt(fmt),
                                             _stream(stream))
    _check("razer_quantize_weights_batch", st)
    return codes, scales, ts[:n]


def razer_quantize_acts(X: torch.Tensor, ts_in: torch.Tensor | None = None, fmt="act", *, hist: bool = True,
                        codes=None, scales=None, ts_out=None, meta_hist=None, stream=None):
    """Quantize activations X [M, K]. ts_in (device f32 [1]) = static scale,
    None = dynamic. Returns (codes, scales, ts_out, meta_hist [4] i64 or None)."""
    M, K = X.shape
    dev = X.device
    codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev) if codes is None else codes
    scales = torch.empty((M, K // 16), dtype=torch.uint8, device=dev) if scales is None else scales
    ts_out = torch.empty(1, dtype=torch.float32, device=dev) if ts_out is None else ts_out
    if hist and meta_hist is None:
        meta_hist = torch.empty(4, dtype=torch.int64, device=dev)
    st = load().razer_quantize_acts(_p(X), _DT.get(X.dtype, -1), M, K, _p(ts_in), _p(codes), _p(scales), _p(ts_out),
                                    _p(meta_hist) if hist else None, _fmt(fmt), _stream(stream))
    _check("razer_quantize_acts", st)
    return codes, scales, ts_out, (meta_hist if hist else None)


def razer_dequant(codes: torch.Tensor, scales: torch.Tensor, ts: torch.Tensor, fmt="weight",
                  out_dtype=torch.float32, *, out=None, stream=None):
    R, K2 = codes.shape
    K = 2 * K2
    out = torch.empty((R, K), dtype=out_dtype, device=codes.device) if out is None else out
    st = load().razer_dequant(_p(codes), _p(scales), _p(ts), _fmt(fmt), R, K, _p(out), _DT.get(out.dtype, -1), _stream(stream))
    _check("razer_dequant", st)
    return out


def razer_workspace_size(op: int, m_or_b: int, N: int, K: int) -> int:
    return int(load().razer_workspace_size(op, m_or_b, N, K))


def _workspace(op, m, N, K, dev, workspace):
    need = razer_workspace_size(op, m, N, K)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    return workspace, (workspace.numel() * workspace.element_size() if workspace is not None else 0)


def razer_gemv(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, ts: torch.Tensor, fmt="weight",
               out_dtype=torch.float32, *, out=None, workspace=None, stream=None):
    """y [B, N] = ts * x [B, K] . deq(W [N, K])^T with 1 <= B <= 32."""
    B, K = x.shape
    N = codes.shape[0]
    out = torch.empty((B, N), dtype=out_dtype, device=x.device) if out is None else out
    workspace, wsb = _workspace(RAZER_OP_GEMV, B, N, K, x.device, workspace)
    st = load().razer_gemv(_p(x), _DT.get(x.dtype, -1), B, _p(codes), _p(scales), _p(ts), _fmt(fmt), N, K, _p(out),
                           _DT.get(out.dtype, -1), _p(workspace), wsb, _stream(stream))
    _check("razer_gemv", st)
    return out


def razer_gemm_w4a4(codes_a: torch.Tensor, scales_a: torch.Tensor, ts_a: torch.Tensor, codes_w: torch.Tensor,
                    scales_w: torch.Tensor, ts_w: torch.Tensor, afmt="act", wfmt="weight", out_dtype=torch.bfloat16, *,
                    out=None, workspace=None, stream=None):
    """Y [M, N] = ts_a * ts_w * deq(A [M, K]) . deq(W [N, K])^T, both operands RaZeR-packed."""
    M, N, K = codes_a.shape[0], codes_w.shape[0], codes_w.shape[1] * 2
    dev = codes_w.device
    out = torch.empty((M, N), dtype=out_dtype, device=dev) if out is None else out
    workspace, wsb = _workspace(RAZER_OP_GEMM_W4A4, M, N, K, dev, workspace)
    st = load().razer_gemm_w4a4(_p(codes_a), _p(scales_a), _p(ts_a), _fmt(afmt), M, _p(codes_w), _p(scales_w), _p(ts_w),
                                _fmt(wfmt), N, K, _p(out), _DT.get(out.dtype, -1), _p(workspace), wsb, _stream(stream))
    _check("razer_gemm_w4a4", st)
    return out


def razer_gemm_w4a4_online(X: torch.Tensor, codes_w: torch.Tensor, scales_w: torch.Tensor, ts_w: torch.Tensor,
                           ts_in: torch.Tensor | None = None, afmt="act", wfmt="weight", out_dtype=torch.bfloat16, *,
                           keep_codes: bool = False, hist: bool = False, out=None, workspace=None, stream=None):
    """Quantize activations X [M, K] and multiply with the packed weights W [N, K]
    in one call. Returns (Y [M, N], ts_a [1], (codes_a, scales_a) or None, meta_hist or None)."""
    M, K = X.shape
    N = codes_w.shape[0]
    dev = X.device
    out = torch.empty((M, N), dtype=out_dtype, device=dev) if out is None else out
    ts_a = torch.empty(1, dtype=torch.float32, device=dev)
    ca = torch.empty((M, K // 2), dtype=torch.uint8, device=dev) if keep_codes else None
    sa = torch.empty((M, K // 16), dtype=torch.uint8, device=dev) if keep_codes else None
    mh = torch.empty(4, dtype=torch.int64, device=dev) if hist else None
    workspace, wsb = _workspace(RAZER_OP_GEMM_W4A4, M, N, K, dev, workspace)
    st = load().razer_gemm_w4a4_online(_p(X), _DT.get(X.dtype, -1), M, _p(ts_in), _fmt(afmt), _p(ca), _p(sa), _p(ts_a), _p(mh),
                                       _p(codes_w), _p(scales_w), _p(ts_w), _fmt(wfmt), N, K, _p(out), _DT.get(out.dtype, -1),
                                       _p(workspace), wsb, _stream(stream))
    _check("razer_gemm_w4a4_online", st)
    return out, ts_a, ((ca, sa) if keep_codes else None), mh


def _varr(V):
    return (ctypes.c_float * max(len(V), 1))(*[float(v) for v in V])


def razer_quantize_variant(X: torch.Tensor, block: int, scale_fmt, V, *, stream=None):
    """RaZeR quantization with a `block`-element block and special values V.
    Returns (codes [R, K/2], scales [R, K/block], ts [1])."""
    R, K = X.shape
    dev = X.device
    codes = torch.empty((R, K // 2), dtype=torch.uint8, device=dev)
    wide = _fmt(scale_fmt) == RAZER_SCALE_F16
    scales = torch.empty((R, (K // block) * (2 if wide else 1)), dtype=torch.uint8, device=dev)
    ts = torch.empty(1, dtype=torch.float32, device=dev)
    st = load().razer_quantize_variant(_p(X), _DT.get(X.dtype, -1), R, K, block, _fmt(scale_fmt), _varr(V), len(V), _p(codes),
                                       _p(scales), _p(ts), _stream(stream))
    _check("razer_quantize_variant", st)
    return codes, scales, ts


def razer_dequant_variant(codes: torch.Tensor, scales: torch.Tensor, ts: torch.Tensor, block: int, scale_fmt, V,
                          out_dtype=torch.float32, *, out=None, stream=None):
    """Decode a razer_quantize_variant tensor to [R, K]: (q*s)*ts rounded once to out_dtype."""
    R, K2 = codes.shape
    K = 2 * K2
    out = torch.empty((R, K), dtype=out_dtype, device=codes.device) if out is None else out
    st = load().razer_dequant_variant(_p(codes), _p(scales), _p(ts), R, K, block, _fmt(scale_fmt), _varr(V), len(V), _p(out),
                                      _DT.get(out.dtype, -1), _stream(stream))
    _check("razer_dequant_variant", st)
    return out


def razer_gemv_variant(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, ts: torch.Tensor, block: int, scale_fmt, V,
                       out_dtype=torch.float32, *, out=None, workspace=None, stream=None):
    """y [B, N] = ts * x [B, K] . deq(W [N, K])^T for a razer_quantize_variant weight tensor, 1 <= B <= 32."""
    B, K = x.shape
    N = codes.shape[0]
    out = torch.empty((B, N), dtype=out_dtype, device=x.device) if out is None else out
    workspace, wsb = _workspace(RAZER_OP_GEMV, B, N, K, x.device, workspace)
    st = load().razer_gemv_variant(_p(x), _DT.get(x.dtype, -1), B, _p(codes), _p(scales), _p(ts), block, _fmt(scale_fmt),
                                   _varr(V), len(V), N, K, _p(out), _DT.get(out.dtype, -1), _p(workspace), wsb, _stream(stream))
    _check("razer_gemv_variant", st)
    return out


def razer_gemm_variant(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, ts: torch.Tensor, block: int, scale_fmt, V,
                       out_dtype=torch.bfloat16, *, out=None, workspace=None, stream=None):
    """Y [M, N] = ts * X [M, K] . deq(W [N, K])^T for a razer_quantize_variant weight tensor (tcgen05 GEMM)."""
    M, K = X.shape
    N = codes.shape[0]
    out = torch.empty((M, N), dtype=out_dtype, device=X.device) if out is None else out
    workspace, wsb = _workspace(RAZER_OP_GEMM_VARIANT, M, N, K, X.device, workspace)
    st = load().razer_gemm_variant(_p(X), _DT.get(X.dtype, -1), M, _p(codes), _p(scales), _p(ts), block, _fmt(scale_fmt),
                                   _varr(V), len(V), N, K, _p(out), _DT.get(out.dtype, -1), _p(workspace), wsb, _stream(stream))
    _check("razer_gemm_variant", st)
    return out


def razer_quant_error_variant(X: torch.Tensor, block: int, scale_fmt, V, codes, scales, ts, *, out=None, stream=None):
    """sum (X - deq(X))^2 (double, device [1]) for a tensor of razer_quantize_variant."""
    R, K = X.shape
    out = torch.empty(1, dtype=torch.float64, device=X.device) if out is None else out
    st = load().razer_quant_error_variant(_p(X), _DT.get(X.dtype, -1), R, K, block, _fmt(scale_fmt), _varr(V), len(V), _p(codes),
                                          _p(scales), _p(ts), _p(out), _stream(stream))
    _check("razer_quant_error_variant", st)
    return out


def razer_quant_error(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, ts: torch.Tensor, fmt="weight", *,
                      out=None, stream=None) -> torch.Tensor:
    """sum (X - deq(X))^2 over the tensor in double (device [1] f64)."""
    R, K = X.shape
    out = torch.empty(1, dtype=torch.float64, device=X.device) if out is None else out
    st = load().razer_quant_error(_p(X), _DT.get(X.dtype, -1), R, K, _p(codes), _p(scales), _p(ts), _fmt(fmt), _p(out),
                                  _stream(stream))
    _check("razer_quant_error", st)
    return out


def razer_gemv_batch(problems, fmt="weight", out_dtype=torch.float32, *, outs=None, workspace=None, stream=None):
    """Several independent GEMVs in one call: problems = [(x, codes, scales,
    ts), ...] (same activation dtype and device). Returns [y_i [B_i, N_i]]."""
    n = len(problems)
    if n == 0:
        return []
    dev = problems[0][0].device
    outs = [torch.empty((x.shape[0], c.shape[0]), dtype=out_dtype, device=dev) for x, c, _, _ in problems] if outs is None else outs
    arr = (GemvProblem * n)(*[GemvProblem(x.data_ptr(), x.shape[0], c.data_ptr(), s.data_ptr(), t.data_ptr(), c.shape[0], x.shape[1],
                                          y.data_ptr()) for (x, c, s, t), y in zip(problems, outs)])
    L = load()
    need = int(L.razer_gemv_batch_workspace_size(n, arr))
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = L.razer_gemv_batch(n, arr, _DT.get(problems[0][0].dtype, -1), _fmt(fmt), _DT.get(out_dtype, -1), _p(workspace), wsb,
                            _stream(stream))
    _check("razer_gemv_batch", st)
    return outs


def razer_gemv_batch_workspace_size(problems) -> int:
    """Workspace bytes razer_gemv_batch needs for problems [(x, codes, scales, ts), ...]."""
    n = len(problems)
    arr = (GemvProblem * max(n, 1))(*[GemvProblem(x.data_ptr(), x.shape[0], c.data_ptr(), s.data_ptr(), t.data_ptr(), c.shape[0],
                                                  x.shape[1], 0) for x, c, s, t in problems])
    return int(load().razer_gemv_batch_workspace_size(n, arr))


def razer_gemv_noalloc(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, ts: torch.Tensor, fmt="weight",
                       out_dtype=torch.float32, *, out=None, stream=None):
    """razer_gemv without a workspace: the split-K scratch is a fixed array
    inside the library (for callers that cannot allocate device memory)."""
    B, K = x.shape
    N = codes.shape[0]
    out = torch.empty((B, N), dtype=out_dtype, device=x.device) if out is None else out
    st = load().razer_gemv_noalloc(_p(x), _DT.get(x.dtype, -1), B, _p(codes), _p(scales), _p(ts), _fmt(fmt), N, K,
                                   _p(out), _DT.get(out.dtype, -1), _stream(stream))
    _check("razer_gemv_noalloc", st)
    return out


def razer_gemv_noalloc_max_scratch() -> int:
    return int(load().razer_gemv_noalloc_max_scratch())


def razer_gemm(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, ts: torch.Tensor, fmt="weight",
               out_dtype=torch.bfloat16, *, out=None, workspace=None, stream=None):
    """Y [M, N] = ts * X [M, K] . deq(W [N, K])^T on the tcgen05 tensor cores."""
    M, K = X.shape
    N = codes.shape[0]
    out = torch.empty((M, N), dtype=out_dtype, device=X.device) if out is None else out
    workspace, wsb = _workspace(RAZER_OP_GEMM, M, N, K, X.device, workspace)
    st = load().razer_gemm(_p(X), _DT.get(X.dtype, -1), M, _p(codes), _p(scales), _p(ts), _fmt(fmt), N, K, _p(out),
                           _DT.get(out.dtype, -1), _p(workspace), wsb, _stream(stream))
    _check("razer_gemm", st)
    return out


# ---- microscaled 4-bit operands (MXFP4, NVFP4) on the block-scaled tensor cores ----
# Scale tiles are uint8 tensors [..., tile rows, tile columns, 512]; include/razer.h
# gives their layout and that of row groups.

_U8, _I32, _F32 = torch.uint8, torch.int32, torch.float32
# torch.cuda.current_stream() builds an object, 3 us: as much as a launch
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _mx_bad(fn: str, name: str, t, shape, dtype, dev: int):
    got = "None" if t is None else f"{tuple(t.shape)} {t.dtype} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}"
    raise ValueError(f"{fn}: {name} must be a contiguous {tuple(shape)} {dtype or ''} tensor on cuda:{max(dev, 0)}, got {got}")


def _mx_ptr(fn: str, name: str, t, shape, dtype, dev: int) -> int:
    """Address of t, a contiguous tensor of this shape, type and device (the library sees only the address)."""
    if t is None or t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _mx_bad(fn, name, t, shape, dtype, dev)
    return t.data_ptr()


def _mx_first(fn: str, name: str, x, dims: int):
    """(shape, device index) of the tensor that sets a call's device: contiguous, of so many dimensions, on a GPU."""
    shape, dev = x.shape, x.get_device()
    if len(shape) != dims or dev < 0 or not x.is_contiguous():
        _mx_bad(fn, name, x, (f"{dims}-dimensional",), None, dev)
    return shape, dev


def _mx_call(fn: str, call, dev: int, *args):
    """Calls the library with dev current, on dev's current stream."""
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _mx_call(fn, call, dev, *args)
    st = call(*args, _raw_stream(dev))
    if st:
        raise RazerError(fn, st)


def _mx_on(fn: str, stream, t, call):
    """call() with stream current: what it allocates then belongs to that stream."""
    if stream.device != t.device:
        raise ValueError(f"{fn}: a stream of {stream.device} for tensors on {t.device}")
    with torch.cuda.stream(stream):
        return call()


def _mx_groups(fn: str, offsets, dev: int) -> tuple[int, int]:
    """(address of the offsets, number of row groups)."""
    shape = offsets.shape
    if len(shape) != 1 or shape[0] < 2:
        raise ValueError(f"{fn}: offsets must hold one entry more than there are groups, and a group at least")
    return _mx_ptr(fn, "offsets", offsets, shape, _I32, dev), shape[0] - 1


def _mx_format(fn: str, fmt) -> tuple[int, int]:
    """(format, elements per block) of a format that has scale tiles; others are left to the library."""
    f = FORMATS[fmt] if isinstance(fmt, str) else int(fmt)
    return f, 16 if f == RAZER_FMT_NVFP4 else 32


def razer_scale_tiles_shape(R: int, K: int, fmt="mxfp4", groups: int = 0) -> tuple[int, int, int]:
    """Shape of the scale tiles of [R, K] codes, or of R rows in `groups` row groups."""
    per = 4 * _mx_format("razer_scale_tiles_shape", fmt)[1]
    return (R // 128 + groups if groups else (R + 127) // 128, (K + per - 1) // per, 512)


def razer_quantize_mx(X: torch.Tensor, offsets: torch.Tensor | None = None, *, codes=None, scales=None, stream=None):
    """Quantize X [M, K] (fp16/bf16, weights or activations) to MXFP4.  Returns
    (codes [M, K/2] u8, scale tiles u8).  offsets (int32 [E + 1], device): rows
    in E groups, as razer_gemm_mx_grouped takes them; rows of no group are left out."""
    fn = "razer_quantize_mx"
    if stream is not None:
        return _mx_on(fn, stream, X, lambda: razer_quantize_mx(X, offsets, codes=codes, scales=scales))
    (M, K), dev = _mx_first(fn, "X", X, 2)
    op, E = (None, 0) if offsets is None else _mx_groups(fn, offsets, dev)
    rows, cols = M // 128 + E if E else (M + 127) // 128, (K + 127) // 128
    if codes is None:
        codes = torch.empty(M, K // 2, dtype=_U8, device=X.device)
        cp = codes.data_ptr()
    else:
        cp = _mx_ptr(fn, "codes", codes, (M, K // 2), _U8, dev)
    if scales is None:
        scales = torch.empty(rows, cols, 512, dtype=_U8, device=X.device)
        sp = scales.data_ptr()
    else:
        sp = _mx_ptr(fn, "scales", scales, (rows, cols, 512), _U8, dev)
    _mx_call(fn, load().razer_quantize_mx, dev, X.data_ptr(), _DT.get(X.dtype, -1), M, K, op, E, cp, sp)
    return codes, scales


def razer_dequant_mx(codes: torch.Tensor, scales: torch.Tensor, out_dtype=torch.float32, offsets: torch.Tensor | None = None, *,
                     out=None, stream=None):
    """Decode MXFP4 codes [M, K/2] with their scale tiles to [M, K] (one rounding to out_dtype)."""
    fn = "razer_dequant_mx"
    if stream is not None:
        return _mx_on(fn, stream, codes, lambda: razer_dequant_mx(codes, scales, out_dtype, offsets, out=out))
    (M, K2), dev = _mx_first(fn, "codes", codes, 2)
    if codes.dtype is not _U8:
        _mx_bad(fn, "codes", codes, codes.shape, _U8, dev)
    op, E = (None, 0) if offsets is None else _mx_groups(fn, offsets, dev)
    sp = _mx_ptr(fn, "scales", scales, (M // 128 + E if E else (M + 127) // 128, (K2 + 63) // 64, 512), _U8, dev)
    if out is None:
        out = torch.empty(M, 2 * K2, dtype=out_dtype, device=codes.device)
    else:
        _mx_ptr(fn, "out", out, (M, 2 * K2), out.dtype, dev)
    _mx_call(fn, load().razer_dequant_mx, dev, codes.data_ptr(), sp, M, 2 * K2, op, E, out.data_ptr(), _DT.get(out.dtype, -1))
    return out


def razer_tile_scales(scales: torch.Tensor, offsets: torch.Tensor | None = None, *, out=None, stream=None):
    """Row-major scale bytes [R, C] or [B, R, C] (as the NVFP4 quantizers write
    them) to scale tiles [..., tile rows, ceil(C/4), 512]; offsets: R rows in groups."""
    fn = "razer_tile_scales"
    if stream is not None:
        return _mx_on(fn, stream, scales, lambda: razer_tile_scales(scales, offsets, out=out))
    dims = 2 if offsets is not None or len(scales.shape) != 3 else 3
    shape, dev = _mx_first(fn, "scales", scales, dims)
    if scales.dtype is not _U8:
        _mx_bad(fn, "scales", scales, shape, _U8, dev)
    op, E = (None, 0) if offsets is None else _mx_groups(fn, offsets, dev)
    R, C = shape[-2:]
    tiles = (R // 128 + E if E else (R + 127) // 128, (C + 3) // 4, 512)
    if dims == 3:
        tiles = (shape[0], *tiles)
    if out is None:
        out = torch.empty(*tiles, dtype=_U8, device=scales.device)
        to = out.data_ptr()
    else:
        to = _mx_ptr(fn, "out", out, tiles, _U8, dev)
    _mx_call(fn, load().razer_tile_scales, dev, scales.data_ptr(), shape[0] if dims == 3 else 1, R, C, op, E, to)
    return out


def _mx_act(fn: str, act) -> int:
    if act not in ACTS:
        raise ValueError(f"{fn}: unknown act {act!r}")
    return ACTS[act]


def _mx_weights(fn: str, codes_w, scales_w, E: int, K2: int, block: int, dev: int):
    """Checks packed weights [N, K/2], or [E, N, K/2] for row groups; returns N and their addresses."""
    shape = codes_w.shape
    if len(shape) != (3 if E else 2) or shape[-1] != K2 or (E and shape[0] != E):
        raise ValueError(f"{fn}: codes_w must be {f'[{E}, N, {K2}]' if E else f'[N, {K2}]'}, got {tuple(shape)}")
    N = shape[-2]
    tiles = ((N + 127) // 128, (2 * K2 + 4 * block - 1) // (4 * block), 512)
    return N, _mx_ptr(fn, "codes_w", codes_w, shape, _U8, dev), _mx_ptr(fn, "scales_w", scales_w, (E, *tiles) if E else tiles, _U8, dev)


def _mx_out(fn: str, out, rows: int, cols: int, out_dtype, like, E: int, dev: int):
    if out is None:  # rows of no group are not written
        return (torch.zeros if E else torch.empty)(rows, cols, dtype=out_dtype, device=like.device)
    _mx_ptr(fn, "out", out, (rows, cols), out.dtype, dev)
    return out


def _mx_product(fn, call, codes_a, scales_a, offsets, codes_w, scales_w, fmt, out_dtype, ts_a, ts_w, act, out, stream):
    if stream is not None:
        return _mx_on(fn, stream, codes_a, lambda: _mx_product(fn, call, codes_a, scales_a, offsets, codes_w, scales_w, fmt, out_dtype, ts_a,
                                                               ts_w, act, out, None))
    (T, K2), dev = _mx_first(fn, "codes_a", codes_a, 2)
    if codes_a.dtype is not _U8:
        _mx_bad(fn, "codes_a", codes_a, (T, K2), _U8, dev)
    f, block = _mx_format(fn, fmt)
    op, E = (None, 0) if offsets is None else _mx_groups(fn, offsets, dev)
    a = _mx_act(fn, act) if act else 0
    sa = _mx_ptr(fn, "scales_a", scales_a, (T // 128 + E if E else (T + 127) // 128, (2 * K2 + 4 * block - 1) // (4 * block), 512), _U8, dev)
    ta = None if ts_a is None else _mx_ptr(fn, "ts_a", ts_a, (1,), _F32, dev)
    tw = None if ts_w is None else _mx_ptr(fn, "ts_w", ts_w, (E or 1,), _F32, dev)
    N, cw, sw = _mx_weights(fn, codes_w, scales_w, E, K2, block, dev)
    out = _mx_out(fn, out, T, N // 2 if a else N, out_dtype, codes_a, E, dev)
    if E:
        _mx_call(fn, call, dev, codes_a.data_ptr(), sa, ta, T, op, E, cw, sw, tw, f, N, 2 * K2, a, out.data_ptr(), _DT.get(out.dtype, -1))
    else:
        _mx_call(fn, call, dev, codes_a.data_ptr(), sa, ta, T, cw, sw, tw, f, N, 2 * K2, a, out.data_ptr(), _DT.get(out.dtype, -1))
    return out


def razer_gemm_mx(codes_a: torch.Tensor, scales_a: torch.Tensor, codes_w: torch.Tensor, scales_w: torch.Tensor, fmt="mxfp4",
                  out_dtype=torch.bfloat16, *, ts_a=None, ts_w=None, act=None, out=None, stream=None):
    """Y [M, N] = ts_a * ts_w * deq(A [M, K]) . deq(W [N, K])^T of packed operands
    (codes and scale tiles; fmt "mxfp4" or "nvfp4") on the block-scaled tensor
    cores.  act="silu_mul": W's rows alternate gate and up, Y [M, N/2]."""
    return _mx_product("razer_gemm_mx", load().razer_gemm_mx, codes_a, scales_a, None, codes_w, scales_w, fmt, out_dtype, ts_a, ts_w, act, out,
                       stream)


def razer_gemm_mx_grouped(codes_a: torch.Tensor, scales_a: torch.Tensor, offsets: torch.Tensor, codes_w: torch.Tensor,
                          scales_w: torch.Tensor, fmt="mxfp4", out_dtype=torch.bfloat16, *, ts_a=None, ts_w=None, act=None, out=None,
                          stream=None):
    """razer_gemm_mx with a weight matrix per row group: rows offsets[e] ..
    offsets[e+1] - 1 of A [T, K] times W[e] of [E, N, K] (ts_w: [E]).  Rows of
    no group are not written (zeros, where the output is made here)."""
    if offsets is None:
        raise ValueError("razer_gemm_mx_grouped: offsets are needed")
    return _mx_product("razer_gemm_mx_grouped", load().razer_gemm_mx_grouped, codes_a, scales_a, offsets, codes_w, scales_w, fmt, out_dtype, ts_a,
                       ts_w, act, out, stream)


@functools.lru_cache(maxsize=1024)
def razer_gemm_mx_grouped_workspace_size(T: int, K: int, groups: int) -> int:
    """Workspace bytes of razer_gemm_mx_grouped_online (groups = 0: of razer_gemm_mx_online)."""
    return int(load().razer_gemm_mx_grouped_workspace_size(T, K, groups))


def _mx_online(fn, call, X, offsets, codes_w, scales_w, out_dtype, act, out, workspace, stream):
    if stream is not None:
        return _mx_on(fn, stream, X, lambda: _mx_online(fn, call, X, offsets, codes_w, scales_w, out_dtype, act, out, workspace, None))
    (T, K), dev = _mx_first(fn, "X", X, 2)
    op, E = (None, 0) if offsets is None else _mx_groups(fn, offsets, dev)
    a = _mx_act(fn, act) if act else 0
    N, cw, sw = _mx_weights(fn, codes_w, scales_w, E, K // 2, 32, dev)
    out = _mx_out(fn, out, T, N // 2 if a else N, out_dtype, X, E, dev)
    if workspace is None:
        ws, wp = razer_gemm_mx_grouped_workspace_size(T, K, E), None
        if ws:
            workspace = torch.empty(ws, dtype=_U8, device=X.device)
            wp = workspace.data_ptr()
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be a contiguous tensor on {X.device}")
    else:
        ws, wp = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    dt = _DT.get(X.dtype, -1)
    if E:
        _mx_call(fn, call, dev, X.data_ptr(), dt, T, op, E, cw, sw, N, K, a, out.data_ptr(), _DT.get(out.dtype, -1), wp, ws)
    else:
        _mx_call(fn, call, dev, X.data_ptr(), dt, T, cw, sw, N, K, a, out.data_ptr(), _DT.get(out.dtype, -1), wp, ws)
    return out


def razer_gemm_mx_online(X: torch.Tensor, codes_w: torch.Tensor, scales_w: torch.Tensor, out_dtype=torch.bfloat16, *, act=None, out=None,
                         workspace=None, stream=None):
    """Quantize X [M, K] (fp16/bf16) to MXFP4 and multiply it with MXFP4 weights
    in one call; equals razer_quantize_mx followed by razer_gemm_mx."""
    return _mx_online("razer_gemm_mx_online", load().razer_gemm_mx_online, X, None, codes_w, scales_w, out_dtype, act, out, workspace, stream)


def razer_gemm_mx_grouped_online(X: torch.Tensor, offsets: torch.Tensor, codes_w: torch.Tensor, scales_w: torch.Tensor,
                                 out_dtype=torch.bfloat16, *, act=None, out=None, workspace=None, stream=None):
    """razer_quantize_mx and razer_gemm_mx_grouped in one call, X [T, K] (fp16/bf16)."""
    if offsets is None:
        raise ValueError("razer_gemm_mx_grouped_online: offsets are needed")
    return _mx_online("razer_gemm_mx_grouped_online", load().razer_gemm_mx_grouped_online, X, offsets, codes_w, scales_w, out_dtype, act, out,
                      workspace, stream)


def razer_get_device_status(stream=None) -> int:
    """Synchronises the stream; returns and clears the device error word."""
    return int(load().razer_get_device_status(_stream(stream)))


def razer_status_string(status: int) -> str:
    return load().razer_status_string(status).decode()


def razer_version() -> int:
    return int(load().razer_version())


RAZER_QPATH_TWO_PASS, RAZER_QPATH_SINGLE_PASS = 0, 1
QUANTIZE_PATHS = {"two_pass": RAZER_QPATH_TWO_PASS, "single_pass": RAZER_QPATH_SINGLE_PASS}


def razer_set_quantize_path(path: str) -> str:
    """Selects the dynamic-scale quantizer path ("two_pass", the default, or
    "single_pass"); returns the previous one."""
    if path not in QUANTIZE_PATHS:
        raise ValueError(f"unknown quantizer path {path!r}")
    prev = int(load().razer_set_quantize_path(QUANTIZE_PATHS[path]))
    return "single_pass" if prev == RAZER_QPATH_SINGLE_PASS else "two_pass"


def razer_debug_set_fault_injection(on: bool) -> bool:
    """Test-only: turns the GEMV / GEMM / single-pass quantizer stall
    injection on or off; returns the previous setting."""
    return bool(load().razer_debug_set_fault_injection(1 if on else 0))
