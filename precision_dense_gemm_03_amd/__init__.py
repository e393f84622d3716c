"""Python binding of libgemm (include/libgemm.h): argument marshalling only.

Every step of the GEMM path runs in the HIP kernels of libgemm.so; this module
only turns torch tensors (device memory) and streams into the C-ABI's plain
pointers and sizes, and turns negative statuses into exceptions. It has no
fallback: if libgemm.so is not built, every call raises.

Functions keep the C names:
    gemm_f16(A, B, C, stream=None)
    gemm_fp8_scaled(A, B, sA, sB, C, sOut=None, stream=None, out_fmt=None)
    gemm_fp8_fmt(A, fmt_a, B, fmt_b, sA, sB, C, sOut=None, stream=None, out_fmt=None)
    quantize_fp8(x, scale, q=None, stream=None) -> q
    quantize_fp8_fmt(x, scale, fmt, q=None, stream=None) -> q
    amax_f32(x, amax=None, scale=None, stream=None) -> (amax, scale)
    amax_scale_f32(x, fmt, pow2, amax=None, scale=None, stream=None) -> (amax, scale)
    gemm_fp8_channel(A, fmt_a, B, fmt_b, sA, sB, C, sOut=None, stream=None, out_fmt=None)
    quantize_fp8_channel(x, scale, axis, fmt, q=None, stream=None) -> q
    amax_scale_channel_f32(x, axis, fmt, pow2, amax=None, scale=None, stream=None) -> (amax, scale)
    gemm_fp8_splitk(A, fmt_a, B, fmt_b, sA, sB, C, sOut=None, workspace=None, stream=None, out_fmt=None)
    gemm_fp8_splitk_noalloc(A, fmt_a, B, fmt_b, sA, sB, C, sOut=None, stream=None, out_fmt=None)
    gemm_f16_splitk(A, B, C, workspace=None, stream=None)
    splitk_plan(kind, out_dtype, M, N, K, fmt_a=0, fmt_b=0) -> (config, splits, workspace_bytes)
    gemm_f16_guarded(A, B, C, scale=None, workspace=None, stream=None) -> (C, scale)
    guarded_workspace_size(M, N, K) -> int
    select_config(kind, out_dtype, M, N, K) -> str   (host-only query)
    select_config_fmt(kind, out_dtype, M, N, K, fmt_a, fmt_b) -> str
  K-major B (Bt[N,K], the layout of a linear layer's weight):
    gemm_f16_bt(A, Bt, C, stream=None)
    gemm_fp8_scaled_bt(A, Bt, sA, sB, C, sOut=None, stream=None, out_fmt=None)
    quantize_fp8_transposed(x, scale, q=None, stream=None) -> q[cols, rows]
    gemm_fp8_fmt_bt(A, fmt_a, Bt, fmt_b, sA, sB, C, sOut=None, stream=None, out_fmt=None)
    quantize_fp8_transposed_fmt(x, scale, fmt, q=None, stream=None) -> q[cols, rows]
    pack_b_kmajor(B, Bt=None, stream=None) -> Bt[N, K]   (FP16 or FP8 codes)
    select_config_bt(kind, out_dtype, M, N, K) -> str
    gemm_fp8_splitk_bt(A, Bt, sA, sB, C, sOut=None, workspace=None, stream=None, out_fmt=None)
    gemm_f16_splitk_bt(A, Bt, C, workspace=None, stream=None)
    splitk_plan_bt(kind, out_dtype, M, N, K) -> (config, splits, workspace_bytes)
  Both FP8 operands in two launches (amax, scale and quantize of A and B):
    amax_quantize_fp8_pair(xa, xb, fmt=FMT_E4M3, pow2=False, amax=None, scale=None, qa=None, qb=None,
                           workspace=None, stream=None) -> (amax[2], scale[2], qa, qb)
    amax_quantize_fp8_pair_bt(xa, xb, fmt=FMT_E4M3, pow2=False, amax=None, scale=None, qa=None, qbt=None,
                              workspace=None, stream=None) -> (amax[2], scale[2], qa, qbt[N, K])
  Exact-accumulation FP8 (FP8 codes widened to FP16, FP16 matrix cores):
    gemm_fp8_exact(A, fmt_a, B, fmt_b, sA, sB, C, sOut=None, stream=None, out_fmt=None)
    gemm_fp8_exact_bt(A, fmt_a, Bt, fmt_b, sA, sB, C, sOut=None, stream=None, out_fmt=None)
    select_config_exact(out_dtype, M, N, K, fmt_a=0, fmt_b=0, b_kmajor=0) -> str
  Products whose weight depends on the row (offsets int32 [groups + 1]; B one weight per group):
    gemm_f16_grouped(A, B, offsets, C, stream=None)              B[groups, K, N]
    gemm_f16_grouped_bt(A, Bt, offsets, C, stream=None)          Bt[groups, N, K]
    gemm_fp8_grouped(A, fmt_a, B, fmt_b, offsets, sA, sB, C, sOut=None, stream=None, out_fmt=None)
    gemm_fp8_grouped_bt, gemm_fp8_grouped_channel, gemm_fp8_grouped_channel_bt: the same arguments
    gemm_f16_grouped_wgrad(A, B, offsets, C, stream=None)        C[groups, M, N]
    gemm_f16_lora_bt(A, Bt, LA, LB, adapter, lscale, C, workspace=None, stream=None)
    gemm_fp8_lora_bt(A, fmt_a, Bt, fmt_b, sA, sB, X, LA, LB, adapter, lscale, C, workspace=None, stream=None)
    lora_workspace_size(rows, rank) -> int
    select_config_grouped(kind, out_dtype, rows, N, K, groups, fmt_a=0, fmt_b=0, b_kmajor=0) -> str
    select_config_wgrad(out_dtype, rows, M, N, groups) -> str
    select_config_lora(kind, out_dtype, rows, N, K, rank, adapters, fmt_a=0, fmt_b=0) -> str
  Expert routing:
    moe_route_f32(logits, topk, renorm=True, expert=None, weight=None, offsets=None, row=None, token=None,
                  workspace=None, stream=None) -> (expert, weight, offsets, row, token)
    moe_route_backward_f32(logits, expert, weight, dweight, renorm=True, dlogits=None, stream=None) -> dlogits
    moe_route_workspace_size(tokens, experts) -> int
    moe_gather(x, token, y=None, stream=None) -> y
    moe_combine(z, row, weight, y=None, stream=None) -> y
    moe_combine_backward(dy, z, row, weight, dZ=None, dweight=None, stream=None) -> (dZ, dweight)
  A dense layer around its products (types from the tensors; 8-bit values are FP8 codes and scale bytes, uint8 or torch's
  float8_e4m3fn / float8_e5m2 and float8_e8m0fnu, one scale per 32 values of a row):
    rms_norm(x, weight, y, eps=1e-5, residual=None, h=None, scale=None, rstd=None, pow2=False, out_fmt=None,
             stream=None) -> y
    rms_norm_backward(dy, h, weight, rstd, dx=None, dweight=None, dh=None, hscale=None, h_fmt=None, workspace=None,
                      stream=None) -> (dx, dweight)
    rms_norm_backward_workspace_size(rows, width) -> int
    gemm_f16_bias_act(A, B, C, bias=None, act=ACT_NONE, residual=None, Z=None, Zscale=None, z_fmt=None, stream=None)
    gemm_f16_bias_act_bt(A, Bt, C, ...): the same arguments
    gemm_fp8_bias_act(A, fmt_a, B, fmt_b, sA, sB, C, bias=None, act=ACT_NONE, residual=None, Z=None, Zscale=None,
                      channel=False, sOut=None, out_fmt=None, z_fmt=None, stream=None)
    gemm_fp8_bias_act_bt(A, fmt_a, Bt, fmt_b, sA, sB, C, ...): the same arguments
    bias_act_backward(dy, Z, act, dZ=None, dbias=None, Zscale=None, z_fmt=None, workspace=None, stream=None)
        -> (dZ, dbias)
    bias_act_backward_workspace_size(rows, cols) -> int
    quantize_mx_fp8(x, fmt=FMT_E4M3, q=None, scale=None, stream=None) -> (q, scale)
    dequantize_mx_fp8(q, scale, fmt, y, stream=None) -> y
    gemm_mx_wgrad(q, scale, fmt, B, C, offsets=None, q_second=False, stream=None) -> C
    select_config_bias_act(kind, out_dtype, M, N, K, fmt_a=0, fmt_b=0, b_kmajor=0, z_dtype=-1) -> str
    select_config_mx_wgrad(out_dtype, rows, M, N, groups=1, q_second=False) -> str
Outputs and workspaces that these calls allocate belong to the call's stream.
The output dtype of a GEMM is taken from C: float32, float16, or 8-bit codes
(uint8 or torch.float8_e4m3fn: E4M3; torch.float8_e5m2, or uint8 with
out_fmt=FMT_E5M2: E5M2). FP8 operands are uint8 codes or torch float8 tensors.
"""
import ctypes
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libgemm.so")

OUT_F32 = 0
OUT_F16 = 1
OUT_E4M3 = 2
OUT_E5M2 = 3
FMT_E4M3 = 0
FMT_E5M2 = 1
KIND_F16 = 0
KIND_FP8 = 1
AXIS_ROW = 0
AXIS_COL = 1
ACT_NONE = 0
ACT_RELU = 1
ACT_GELU = 2
ACT_GELU_TANH = 3
ACT_SILU = 4

GEMM_OK = 0
STATUS_NAMES = {
    0: "GEMM_OK", -1: "GEMM_ERR_NULL", -2: "GEMM_ERR_DIM", -3: "GEMM_ERR_DTYPE",
    -4: "GEMM_ERR_SCALE", -5: "GEMM_ERR_LAUNCH", -6: "GEMM_ERR_UNSUPPORTED",
    -7: "GEMM_ERR_DEVICE", -8: "GEMM_ERR_ALIAS", -9: "GEMM_ERR_WORKSPACE",
}

_lib = None


class GemmError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({status_str(status)})")


def lib() -> ctypes.CDLL:
    """The loaded libgemm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it first (python __graft_entry__.py build, "
                           "or python precision_dense_gemm_03_amd/_build.py)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.gemm_f16.restype = i32
    L.gemm_f16.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp]
    L.gemm_fp8_scaled.restype = i32
    L.gemm_fp8_scaled.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    L.quantize_fp8.restype = i32
    L.quantize_fp8.argtypes = [vp, i64, vp, vp, vp]
    L.amax_f32.restype = i32
    L.amax_f32.argtypes = [vp, i64, vp, vp, vp]
    L.gemm_status_str.restype = ctypes.c_char_p
    L.gemm_status_str.argtypes = [i32]
    L.gemm_select_config.restype = i32
    L.gemm_select_config.argtypes = [i32, i32, i64, i64, i64, ctypes.c_char_p, i32]
    L.gemm_fp8_fmt.restype = i32
    L.gemm_fp8_fmt.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    L.quantize_fp8_fmt.restype = i32
    L.quantize_fp8_fmt.argtypes = [vp, i64, vp, vp, i32, vp]
    L.amax_scale_f32.restype = i32
    L.amax_scale_f32.argtypes = [vp, i64, vp, vp, i32, i32, vp]
    L.gemm_fp8_channel.restype = i32
    L.gemm_fp8_channel.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    L.amax_scale_channel_f32.restype = i32
    L.amax_scale_channel_f32.argtypes = [vp, i64, i64, i32, vp, vp, i32, i32, vp]
    L.quantize_fp8_channel.restype = i32
    L.quantize_fp8_channel.argtypes = [vp, i64, i64, i32, vp, vp, i32, vp]
    L.gemm_fp8_splitk.restype = i32
    L.gemm_fp8_splitk.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, i32, i64, i64, i64, vp, i64, vp]
    L.gemm_fp8_splitk_noalloc.restype = i32
    L.gemm_fp8_splitk_noalloc.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    L.gemm_fp8_splitk_noalloc_max_bytes.restype = i64
    L.gemm_fp8_splitk_noalloc_max_bytes.argtypes = []
    L.gemm_f16_splitk.restype = i32
    L.gemm_f16_splitk.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, i64, vp]
    L.gemm_splitk_plan.restype = i32
    L.gemm_splitk_plan.argtypes = [i32, i32, i64, i64, i64, i32, i32, ctypes.c_char_p, i32,
                                   ctypes.POINTER(i32), ctypes.POINTER(i64)]
    L.gemm_f16_guarded.restype = i32
    L.gemm_f16_guarded.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, vp, i64, vp]
    L.gemm_f16_guarded_workspace_size.restype = i64
    L.gemm_f16_guarded_workspace_size.argtypes = [i64, i64, i64]
    L.gemm_select_config_fmt.restype = i32
    L.gemm_select_config_fmt.argtypes = [i32, i32, i64, i64, i64, i32, i32, ctypes.c_char_p, i32]
    L.gemm_f16_bt.restype = i32
    L.gemm_f16_bt.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp]
    L.gemm_fp8_scaled_bt.restype = i32
    L.gemm_fp8_scaled_bt.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    L.quantize_fp8_transposed.restype = i32
    L.quantize_fp8_transposed.argtypes = [vp, i64, i64, vp, vp, vp]
    L.gemm_select_config_bt.restype = i32
    L.gemm_select_config_bt.argtypes = [i32, i32, i64, i64, i64, ctypes.c_char_p, i32]
    L.gemm_fp8_fmt_bt.restype = i32
    L.gemm_fp8_fmt_bt.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    L.quantize_fp8_transposed_fmt.restype = i32
    L.quantize_fp8_transposed_fmt.argtypes = [vp, i64, i64, vp, vp, i32, vp]
    L.pack_b_kmajor.restype = i32
    L.pack_b_kmajor.argtypes = [vp, i64, i64, i32, vp, vp]
    L.gemm_fp8_splitk_bt.restype = i32
    L.gemm_fp8_splitk_bt.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i64, i64, vp, i64, vp]
    L.gemm_f16_splitk_bt.restype = i32
    L.gemm_f16_splitk_bt.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, i64, vp]
    L.gemm_splitk_plan_bt.restype = i32
    L.gemm_splitk_plan_bt.argtypes = [i32, i32, i64, i64, i64, ctypes.c_char_p, i32, ctypes.POINTER(i32),
                                      ctypes.POINTER(i64)]
    L.amax_quantize_fp8_pair.restype = i32
    L.amax_quantize_fp8_pair.argtypes = [vp, i64, vp, i64, i32, i32, vp, vp, vp, vp, vp, i64, vp]
    L.amax_quantize_fp8_pair_bt.restype = i32
    L.amax_quantize_fp8_pair_bt.argtypes = [vp, i64, vp, i64, i64, i32, i32, vp, vp, vp, vp, vp, i64, vp]
    L.amax_quantize_fp8_pair_workspace_size.restype = i64
    L.amax_quantize_fp8_pair_workspace_size.argtypes = []
    L.gemm_fp8_exact.restype = i32
    L.gemm_fp8_exact.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    L.gemm_fp8_exact_bt.restype = i32
    L.gemm_fp8_exact_bt.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    L.gemm_select_config_exact.restype = i32
    L.gemm_select_config_exact.argtypes = [i32, i64, i64, i64, i32, i32, i32, ctypes.c_char_p, i32]
    for name in ("gemm_f16_grouped", "gemm_f16_grouped_bt"):
        f = getattr(L, name)
        f.restype = i32
        f.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, i64, vp]
    for name in ("gemm_fp8_grouped", "gemm_fp8_grouped_bt", "gemm_fp8_grouped_channel",
                 "gemm_fp8_grouped_channel_bt"):
        f = getattr(L, name)
        f.restype = i32
        f.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, vp, i32, i64, i64, i64, i64, vp]
    L.gemm_f16_grouped_wgrad.restype = i32
    L.gemm_f16_grouped_wgrad.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, i64, vp]
    L.gemm_f16_lora_bt.restype = i32
    L.gemm_f16_lora_bt.argtypes = [vp] * 7 + [i32] + [i64] * 5 + [vp, i64, vp]
    L.gemm_fp8_lora_bt.restype = i32
    L.gemm_fp8_lora_bt.argtypes = [vp, i32, vp, i32] + [vp] * 8 + [i32] + [i64] * 5 + [vp, i64, vp]
    L.gemm_select_config_grouped.restype = i32
    L.gemm_select_config_grouped.argtypes = [i32, i32, i64, i64, i64, i64, i32, i32, i32, ctypes.c_char_p, i32]
    L.gemm_select_config_wgrad.restype = i32
    L.gemm_select_config_wgrad.argtypes = [i32, i64, i64, i64, i64, ctypes.c_char_p, i32]
    L.gemm_select_config_lora.restype = i32
    L.gemm_select_config_lora.argtypes = [i32, i32, i64, i64, i64, i64, i64, i32, i32, ctypes.c_char_p, i32]
    L.gemm_lora_workspace_size.restype = i64
    L.gemm_lora_workspace_size.argtypes = [i64, i64]
    L.moe_route_f32.restype = i32
    L.moe_route_f32.argtypes = [vp, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, i64, vp]
    L.moe_route_workspace_size.restype = i64
    L.moe_route_workspace_size.argtypes = [i64, i64]
    L.moe_route_backward_f32.restype = i32
    L.moe_route_backward_f32.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp, vp]
    L.moe_gather.restype = i32
    L.moe_gather.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp]
    L.moe_combine.restype = i32
    L.moe_combine.argtypes = [vp, i32, vp, vp, vp, i32, i64, i64, i64, i64, vp]
    L.moe_combine_backward.restype = i32
    L.moe_combine_backward.argtypes = [vp, vp, i32, vp, vp, vp, vp, i64, i64, i64, i64, vp]
    f32 = ctypes.c_float
    L.rms_norm.restype = i32
    L.rms_norm.argtypes = [vp, vp, i32, vp, f32, vp, vp, i32, vp, i32, vp, i64, i64, vp]
    L.rms_norm_backward.restype = i32
    L.rms_norm_backward.argtypes = [vp, vp, i32, vp, vp, i32, vp, vp, vp, vp, i64, i64, vp, i64, vp]
    L.rms_norm_backward_workspace_size.restype = i64
    L.rms_norm_backward_workspace_size.argtypes = [i64, i64]
    for name in ("gemm_f16_bias_act", "gemm_f16_bias_act_bt"):
        f = getattr(L, name)
        f.restype = i32
        f.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, vp, vp, i32, i64, i64, i64, vp]
    for name in ("gemm_fp8_bias_act", "gemm_fp8_bias_act_bt"):
        f = getattr(L, name)
        f.restype = i32
        f.argtypes = [vp, i32, vp, i32, vp, vp, i32, vp, vp, vp, i32, vp, i32, i32, vp, vp, i32, i64, i64, i64, vp]
    L.bias_act_backward.restype = i32
    L.bias_act_backward.argtypes = [vp, i32, vp, vp, i32, i32, vp, vp, i64, i64, vp, i64, vp]
    L.bias_act_backward_workspace_size.restype = i64
    L.bias_act_backward_workspace_size.argtypes = [i64, i64]
    L.quantize_mx_fp8.restype = i32
    L.quantize_mx_fp8.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp]
    L.dequantize_mx_fp8.restype = i32
    L.dequantize_mx_fp8.argtypes = [vp, vp, i32, i64, i64, vp, i32, vp]
    L.gemm_mx_wgrad.restype = i32
    L.gemm_mx_wgrad.argtypes = [vp, vp, i32, vp, vp, vp, i32, i64, i64, i64, i64, i32, vp]
    L.gemm_select_config_bias_act.restype = i32
    L.gemm_select_config_bias_act.argtypes = [i32, i32, i64, i64, i64, i32, i32, i32, i32, ctypes.c_char_p, i32]
    L.gemm_select_config_mx_wgrad.restype = i32
    L.gemm_select_config_mx_wgrad.argtypes = [i32, i64, i64, i64, i64, i32, ctypes.c_char_p, i32]
    _lib = L
    return L


def status_str(status: int) -> str:
    return lib().gemm_status_str(int(status)).decode()


def _check(status: int, what: str):
    if status != GEMM_OK:
        raise GemmError(status, what)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_handle(stream):
    if stream is None:
        torch = _torch()
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libgemm takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libgemm takes contiguous (row-major) tensors")
    return t.data_ptr()


def _out_dtype(C, out_fmt=None):
    torch = _torch()
    if C.dtype == torch.float32:
        return OUT_F32
    if C.dtype == torch.float16:
        return OUT_F16
    if C.dtype == torch.float8_e5m2 or (C.dtype == torch.uint8 and out_fmt == FMT_E5M2):
        return OUT_E5M2
    if C.dtype in (torch.uint8, torch.float8_e4m3fn):
        return OUT_E4M3
    raise ValueError(f"unsupported output dtype {C.dtype}")


def _dims(A, B, C):
    if A.dim() != 2 or B.dim() != 2 or C.dim() != 2:
        raise ValueError("A, B and C must be 2-D")
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    return M, N, K


def _dims_bt(A, Bt, C):
    if A.dim() != 2 or Bt.dim() != 2 or C.dim() != 2:
        raise ValueError("A, Bt and C must be 2-D")
    M, K = A.shape
    N, K2 = Bt.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} Bt{tuple(Bt.shape)} C{tuple(C.shape)}")
    return M, N, K


def gemm_f16_bt(A, Bt, C, stream=None):
    """C = A @ Bt.T for float16 A[M,K] and a K-major weight Bt[N,K]; C float32 or float16 [M,N]."""
    torch = _torch()
    if A.dtype != torch.float16 or Bt.dtype != torch.float16:
        raise ValueError("gemm_f16_bt takes float16 operands")
    M, N, K = _dims_bt(A, Bt, C)
    _check(lib().gemm_f16_bt(_ptr(A), _ptr(Bt), _ptr(C), _out_dtype(C), M, N, K, _stream_handle(stream)),
           "gemm_f16_bt")
    return C


def gemm_f16(A, B, C, stream=None):
    """C = A @ B for float16 A[M,K], B[K,N]; C float32 or float16 [M,N]."""
    torch = _torch()
    if A.dtype != torch.float16 or B.dtype != torch.float16:
        raise ValueError("gemm_f16 takes float16 operands")
    M, N, K = _dims(A, B, C)
    _check(lib().gemm_f16(_ptr(A), _ptr(B), _ptr(C), _out_dtype(C), M, N, K, _stream_handle(stream)), "gemm_f16")
    return C


def _u8(t, fmt=None):
    """The uint8 view of FP8 codes. A torch float8 tensor must be of format
    fmt when one is given (FMT_E4M3 / FMT_E5M2): its bits are not re-encoded."""
    torch = _torch()
    if t.dtype in (torch.float8_e4m3fn, torch.float8_e5m2):
        have = FMT_E5M2 if t.dtype == torch.float8_e5m2 else FMT_E4M3
        if fmt is not None and int(fmt) != have:
            want = "E5M2" if int(fmt) == FMT_E5M2 else "E4M3"
            raise ValueError(f"a {t.dtype} tensor was passed where {want} codes are expected")
        return t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise ValueError("FP8 tensors must be uint8 codes or torch float8 tensors")
    return t


def gemm_fp8_scaled(A, B, sA, sB, C, sOut=None, stream=None, out_fmt=None):
    """C = (sA*A) @ (sB*B) for E4M3 A[M,K], B[K,N]; sA, sB (and sOut for an
    FP8 C) are one-element float32 device tensors."""
    A, B = _u8(A, FMT_E4M3), _u8(B, FMT_E4M3)
    out = _out_dtype(C, out_fmt)
    Cv = _u8(C) if out in (OUT_E4M3, OUT_E5M2) else C
    M, N, K = _dims(A, B, Cv)
    _check(lib().gemm_fp8_scaled(_ptr(A), _ptr(B), _ptr(sA), _ptr(sB), _ptr(sOut), _ptr(Cv), out, M, N, K,
                                 _stream_handle(stream)), "gemm_fp8_scaled")
    return C


def gemm_fp8_scaled_bt(A, Bt, sA, sB, C, sOut=None, stream=None, out_fmt=None):
    """gemm_fp8_scaled with B given K-major: C = (sA*A) @ (sB*Bt).T for E4M3
    A[M,K] and Bt[N,K]."""
    A, Bt = _u8(A, FMT_E4M3), _u8(Bt, FMT_E4M3)
    out = _out_dtype(C, out_fmt)
    Cv = _u8(C) if out in (OUT_E4M3, OUT_E5M2) else C
    M, N, K = _dims_bt(A, Bt, Cv)
    _check(lib().gemm_fp8_scaled_bt(_ptr(A), _ptr(Bt), _ptr(sA), _ptr(sB), _ptr(sOut), _ptr(Cv), out, M, N, K,
                                    _stream_handle(stream)), "gemm_fp8_scaled_bt")
    return C


def gemm_fp8_fmt_bt(A, fmt_a, Bt, fmt_b, sA, sB, C, sOut=None, stream=None, out_fmt=None):
    """gemm_fp8_scaled_bt with A in FP8 format fmt_a and Bt in fmt_b (FMT_E4M3 / FMT_E5M2)."""
    A, Bt = _u8(A, fmt_a), _u8(Bt, fmt_b)
    out = _out_dtype(C, out_fmt)
    Cv = _u8(C) if out in (OUT_E4M3, OUT_E5M2) else C
    M, N, K = _dims_bt(A, Bt, Cv)
    _check(lib().gemm_fp8_fmt_bt(_ptr(A), int(fmt_a), _ptr(Bt), int(fmt_b), _ptr(sA), _ptr(sB), _ptr(sOut), _ptr(Cv),
                                 out, M, N, K, _stream_handle(stream)), "gemm_fp8_fmt_bt")
    return C


def quantize_fp8_transposed_fmt(x, scale, fmt, q=None, stream=None):
    """quantize_fp8_transposed into FP8 format fmt (FMT_E4M3 / FMT_E5M2)."""
    torch = _torch()
    if x.dtype != torch.float32:
        raise ValueError("quantize_fp8_transposed_fmt takes float32 input")
    rows, cols = _rows_cols(x)
    if q is None:
        q = torch.empty((cols, rows), dtype=torch.uint8, device=x.device)
    qv = _u8(q, fmt)
    if qv.numel() != x.numel():
        raise ValueError("q must have as many elements as x")
    _check(lib().quantize_fp8_transposed_fmt(_ptr(x), rows, cols, _ptr(scale), _ptr(qv), int(fmt),
                                             _stream_handle(stream)), "quantize_fp8_transposed_fmt")
    return q


def pack_b_kmajor(B, Bt=None, stream=None):
    """The K-major copy Bt[N, K] of a row-major weight B[K, N] (float16, or
    FP8 codes as uint8 / torch float8), made once on the GPU."""
    torch = _torch()
    if B.dim() != 2:
        raise ValueError("pack_b_kmajor takes a 2-D B")
    es = B.element_size()
    if es not in (1, 2):
        raise ValueError("pack_b_kmajor takes 1- or 2-byte elements")
    K, N = int(B.shape[0]), int(B.shape[1])
    if Bt is None:
        Bt = torch.empty((N, K), dtype=B.dtype, device=B.device)
    if tuple(Bt.shape) != (N, K) or Bt.element_size() != es:
        raise ValueError("Bt must be [N, K] with B's element size")
    _check(lib().pack_b_kmajor(_ptr(B), K, N, es, _ptr(Bt), _stream_handle(stream)), "pack_b_kmajor")
    return Bt


def quantize_fp8_transposed(x, scale, q=None, stream=None):
    """E4M3 codes of x / scale for a 2-D float32 x[rows, cols], written
    transposed: q[cols, rows] (uint8)."""
    torch = _torch()
    if x.dtype != torch.float32:
        raise ValueError("quantize_fp8_transposed takes float32 input")
    rows, cols = _rows_cols(x)
    if q is None:
        q = torch.empty((cols, rows), dtype=torch.uint8, device=x.device)
    qv = _u8(q, FMT_E4M3)
    if qv.numel() != x.numel():
        raise ValueError("q must have as many elements as x")
    _check(lib().quantize_fp8_transposed(_ptr(x), rows, cols, _ptr(scale), _ptr(qv), _stream_handle(stream)),
           "quantize_fp8_transposed")
    return q


def gemm_fp8_fmt(A, fmt_a, B, fmt_b, sA, sB, C, sOut=None, stream=None, out_fmt=None):
    """gemm_fp8_scaled with A in FP8 format fmt_a and B in fmt_b (FMT_E4M3 / FMT_E5M2)."""
    A, B = _u8(A, fmt_a), _u8(B, fmt_b)
    out = _out_dtype(C, out_fmt)
    Cv = _u8(C) if out in (OUT_E4M3, OUT_E5M2) else C
    M, N, K = _dims(A, B, Cv)
    _check(lib().gemm_fp8_fmt(_ptr(A), int(fmt_a), _ptr(B), int(fmt_b), _ptr(sA), _ptr(sB), _ptr(sOut), _ptr(Cv),
                              out, M, N, K, _stream_handle(stream)), "gemm_fp8_fmt")
    return C


def gemm_fp8_channel(A, fmt_a, B, fmt_b, sA, sB, C, sOut=None, stream=None, out_fmt=None):
    """gemm_fp8_fmt with per-channel scales: sA float32[M] (one per row of A),
    sB float32[N] (one per column of B); sOut stays one element."""
    A, B = _u8(A, fmt_a), _u8(B, fmt_b)
    out = _out_dtype(C, out_fmt)
    Cv = _u8(C) if out in (OUT_E4M3, OUT_E5M2) else C
    M, N, K = _dims(A, B, Cv)
    torch = _torch()
    for name, s, n in (("sA", sA, M), ("sB", sB, N)):
        if s.dtype != torch.float32 or s.numel() != n:
            raise ValueError(f"{name} must be float32 with one scale per channel ({n})")
    _check(lib().gemm_fp8_channel(_ptr(A), int(fmt_a), _ptr(B), int(fmt_b), _ptr(sA), _ptr(sB), _ptr(sOut),
                                  _ptr(Cv), out, M, N, K, _stream_handle(stream)), "gemm_fp8_channel")
    return C


def _rows_cols(x):
    if x.dim() != 2:
        raise ValueError("per-channel calls take a 2-D x")
    return int(x.shape[0]), int(x.shape[1])


def quantize_fp8_channel(x, scale, axis, fmt, q=None, stream=None):
    """FP8 codes of x[i,j] / scale[i] (axis AXIS_ROW) or / scale[j] (AXIS_COL)."""
    torch = _torch()
    if x.dtype != torch.float32:
        raise ValueError("quantize_fp8_channel takes float32 input")
    rows, cols = _rows_cols(x)
    if scale.dtype != torch.float32 or scale.numel() != (rows if axis == AXIS_ROW else cols):
        raise ValueError("one float32 scale per channel")
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    qv = _u8(q, fmt)
    if qv.numel() != x.numel():
        raise ValueError("q must have as many elements as x")
    _check(lib().quantize_fp8_channel(_ptr(x), rows, cols, int(axis), _ptr(scale), _ptr(qv), int(fmt),
                                      _stream_handle(stream)), "quantize_fp8_channel")
    return q


def amax_scale_channel_f32(x, axis, fmt, pow2, amax=None, scale=None, stream=None):
    """(amax, scale) per row (axis AXIS_ROW) or per column (AXIS_COL) of x."""
    torch = _torch()
    if x.dtype != torch.float32:
        raise ValueError("amax_scale_channel_f32 takes float32 input")
    rows, cols = _rows_cols(x)
    n = rows if axis == AXIS_ROW else cols
    if amax is None:
        amax = torch.empty(n, dtype=torch.float32, device=x.device)
    if scale is None:
        scale = torch.empty(n, dtype=torch.float32, device=x.device)
    if amax.numel() != n or scale.numel() != n:
        raise ValueError("amax and scale need one element per channel")
    _check(lib().amax_scale_channel_f32(_ptr(x), rows, cols, int(axis), _ptr(amax), _ptr(scale), int(fmt),
                                        1 if pow2 else 0, _stream_handle(stream)), "amax_scale_channel_f32")
    return amax, scale


def splitk_plan(kind: int, out_dtype: int, M: int, N: int, K: int, fmt_a: int = 0, fmt_b: int = 0):
    """(configuration name, number of K ranges, workspace bytes) of the
    split-K entry points for this request (host-only query)."""
    buf = ctypes.create_string_buffer(64)
    sp = ctypes.c_int(0)
    wb = ctypes.c_int64(0)
    _check(lib().gemm_splitk_plan(kind, out_dtype, M, N, K, fmt_a, fmt_b, buf, 64, ctypes.byref(sp),
                                  ctypes.byref(wb)), "gemm_splitk_plan")
    return buf.value.decode(), sp.value, wb.value


def _workspace(kind, out, M, N, K, fa, fb, workspace, device):
    if workspace is not None:
        return workspace
    _, _, nbytes = splitk_plan(kind, out, M, N, K, fa, fb)
    if nbytes == 0:
        return None
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device)


def _ws_args(workspace):
    if workspace is None:
        return None, 0
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def gemm_fp8_splitk(A, fmt_a, B, fmt_b, sA, sB, C, sOut=None, workspace=None, stream=None, out_fmt=None):
    """gemm_fp8_fmt that splits K over a workspace when the shape has too few
    output tiles; workspace=None allocates one of the planned size."""
    A, B = _u8(A, fmt_a), _u8(B, fmt_b)
    out = _out_dtype(C, out_fmt)
    Cv = _u8(C) if out in (OUT_E4M3, OUT_E5M2) else C
    M, N, K = _dims(A, B, Cv)
    ws, nbytes = _ws_args(_workspace(KIND_FP8, out, M, N, K, int(fmt_a), int(fmt_b), workspace, C.device))
    _check(lib().gemm_fp8_splitk(_ptr(A), int(fmt_a), _ptr(B), int(fmt_b), _ptr(sA), _ptr(sB), _ptr(sOut), _ptr(Cv),
                                 out, M, N, K, ws, nbytes, _stream_handle(stream)), "gemm_fp8_splitk")
    return C


def gemm_fp8_splitk_noalloc(A, fmt_a, B, fmt_b, sA, sB, C, sOut=None, stream=None, out_fmt=None):
    """gemm_fp8_splitk with the partial sums in the library's own per-GPU
    array (no workspace, nothing allocated); calls that overlap on one GPU
    race."""
    A, B = _u8(A, fmt_a), _u8(B, fmt_b)
    out = _out_dtype(C, out_fmt)
    Cv = _u8(C) if out in (OUT_E4M3, OUT_E5M2) else C
    M, N, K = _dims(A, B, Cv)
    _check(lib().gemm_fp8_splitk_noalloc(_ptr(A), int(fmt_a), _ptr(B), int(fmt_b), _ptr(sA), _ptr(sB), _ptr(sOut),
                                         _ptr(Cv), out, M, N, K, _stream_handle(stream)), "gemm_fp8_splitk_noalloc")
    return C


def gemm_fp8_splitk_noalloc_max_bytes() -> int:
    return int(lib().gemm_fp8_splitk_noalloc_max_bytes())


def gemm_f16_splitk(A, B, C, workspace=None, stream=None):
    """gemm_f16 that splits K over a workspace when the shape has too few
    output tiles; workspace=None allocates one of the planned size."""
    out = _out_dtype(C)
    if out not in (OUT_F32, OUT_F16):
        raise ValueError("gemm_f16 writes float32 or float16")
    M, N, K = _dims(A, B, C)
    ws, nbytes = _ws_args(_workspace(KIND_F16, out, M, N, K, 0, 0, workspace, C.device))
    _check(lib().gemm_f16_splitk(_ptr(A), _ptr(B), _ptr(C), out, M, N, K, ws, nbytes, _stream_handle(stream)),
           "gemm_f16_splitk")
    return C


def guarded_workspace_size(M: int, N: int, K: int) -> int:
    n = int(lib().gemm_f16_guarded_workspace_size(M, N, K))
    _check(n if n < 0 else 0, "gemm_f16_guarded_workspace_size")
    return n


def gemm_f16_guarded(A, B, C, scale=None, workspace=None, stream=None):
    """C = A @ B for float32 A[M,K], B[K,N] through the FP16 GEMM under the
    dynamic-range guard; returns (C, scale) with scale the one-element s."""
    torch = _torch()
    if A.dtype != torch.float32 or B.dtype != torch.float32:
        raise ValueError("gemm_f16_guarded takes float32 A and B")
    out = _out_dtype(C)
    if out not in (OUT_F32, OUT_F16):
        raise ValueError("gemm_f16_guarded writes float32 or float16")
    M, N, K = _dims(A, B, C)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=C.device)
    if workspace is None:
        workspace = torch.empty(guarded_workspace_size(M, N, K), dtype=torch.uint8, device=C.device)
    _check(lib().gemm_f16_guarded(_ptr(A), _ptr(B), _ptr(C), out, M, N, K, _ptr(scale), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream_handle(stream)),
           "gemm_f16_guarded")
    return C, scale


def quantize_fp8(x, scale, q=None, stream=None):
    """E4M3 codes of x / scale (uint8, same shape as x)."""
    torch = _torch()
    if x.dtype != torch.float32:
        raise ValueError("quantize_fp8 takes float32 input")
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    qv = _u8(q, FMT_E4M3)
    if qv.numel() != x.numel():
        raise ValueError("q must have as many elements as x")
    _check(lib().quantize_fp8(_ptr(x), x.numel(), _ptr(scale), _ptr(qv), _stream_handle(stream)), "quantize_fp8")
    return q


def quantize_fp8_fmt(x, scale, fmt, q=None, stream=None):
    """FP8 codes (format fmt) of x / scale (uint8, same shape as x)."""
    torch = _torch()
    if x.dtype != torch.float32:
        raise ValueError("quantize_fp8_fmt takes float32 input")
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    qv = _u8(q, fmt)
    if qv.numel() != x.numel():
        raise ValueError("q must have as many elements as x")
    _check(lib().quantize_fp8_fmt(_ptr(x), x.numel(), _ptr(scale), _ptr(qv), int(fmt), _stream_handle(stream)),
           "quantize_fp8_fmt")
    return q


def amax_scale_f32(x, fmt, pow2, amax=None, scale=None, stream=None):
    """(amax, scale) with the scale for FP8 format fmt: amax / fmax, or with pow2
    the smallest power of two s with amax / s <= fmax."""
    torch = _torch()
    if x.dtype != torch.float32:
        raise ValueError("amax_scale_f32 takes float32 input")
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=x.device)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(lib().amax_scale_f32(_ptr(x), x.numel(), _ptr(amax), _ptr(scale), int(fmt), 1 if pow2 else 0,
                                _stream_handle(stream)), "amax_scale_f32")
    return amax, scale


def amax_f32(x, amax=None, scale=None, stream=None):
    """(amax, scale): max|x| and max|x|/448 (1 if that is 0) as 1-element device tensors."""
    torch = _torch()
    if x.dtype != torch.float32:
        raise ValueError("amax_f32 takes float32 input")
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=x.device)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(lib().amax_f32(_ptr(x), x.numel(), _ptr(amax), _ptr(scale), _stream_handle(stream)), "amax_f32")
    return amax, scale


def select_config(kind: int, out_dtype: int, M: int, N: int, K: int) -> str:
    buf = ctypes.create_string_buffer(128)
    _check(lib().gemm_select_config(kind, out_dtype, M, N, K, buf, len(buf)), "gemm_select_config")
    return buf.value.decode()


def select_config_fmt(kind: int, out_dtype: int, M: int, N: int, K: int, fmt_a: int, fmt_b: int) -> str:
    buf = ctypes.create_string_buffer(128)
    _check(lib().gemm_select_config_fmt(kind, out_dtype, M, N, K, int(fmt_a), int(fmt_b), buf, len(buf)),
           "gemm_select_config_fmt")
    return buf.value.decode()


def select_config_bt(kind: int, out_dtype: int, M: int, N: int, K: int) -> str:
    """The configuration gemm_f16_bt (kind 0) or gemm_fp8_scaled_bt (kind 1) would launch."""
    buf = ctypes.create_string_buffer(128)
    _check(lib().gemm_select_config_bt(kind, out_dtype, M, N, K, buf, len(buf)), "gemm_select_config_bt")
    return buf.value.decode()


def splitk_plan_bt(kind: int, out_dtype: int, M: int, N: int, K: int):
    """splitk_plan for the K-major split-K calls."""
    buf = ctypes.create_string_buffer(64)
    sp = ctypes.c_int(0)
    wb = ctypes.c_int64(0)
    _check(lib().gemm_splitk_plan_bt(kind, out_dtype, M, N, K, buf, 64, ctypes.byref(sp), ctypes.byref(wb)),
           "gemm_splitk_plan_bt")
    return buf.value.decode(), sp.value, wb.value


def _workspace_bt(kind, out, M, N, K, workspace, device):
    if workspace is not None:
        return workspace
    _, _, nbytes = splitk_plan_bt(kind, out, M, N, K)
    if nbytes == 0:
        return None
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device)


def gemm_fp8_splitk_bt(A, Bt, sA, sB, C, sOut=None, workspace=None, stream=None, out_fmt=None):
    """gemm_fp8_scaled_bt that splits K over a workspace for mid-M shapes;
    workspace=None allocates one of the planned size."""
    A, Bt = _u8(A, FMT_E4M3), _u8(Bt, FMT_E4M3)
    out = _out_dtype(C, out_fmt)
    Cv = _u8(C) if out in (OUT_E4M3, OUT_E5M2) else C
    M, N, K = _dims_bt(A, Bt, Cv)
    ws, nbytes = _ws_args(_workspace_bt(KIND_FP8, out, M, N, K, workspace, C.device))
    _check(lib().gemm_fp8_splitk_bt(_ptr(A), _ptr(Bt), _ptr(sA), _ptr(sB), _ptr(sOut), _ptr(Cv), out, M, N, K, ws,
                                    nbytes, _stream_handle(stream)), "gemm_fp8_splitk_bt")
    return C


def gemm_f16_splitk_bt(A, Bt, C, workspace=None, stream=None):
    """gemm_f16_bt that splits K over a workspace for mid-M shapes."""
    torch = _torch()
    if A.dtype != torch.float16 or Bt.dtype != torch.float16:
        raise ValueError("gemm_f16_splitk_bt takes float16 operands")
    M, N, K = _dims_bt(A, Bt, C)
    out = _out_dtype(C)
    ws, nbytes = _ws_args(_workspace_bt(KIND_F16, out, M, N, K, workspace, C.device))
    _check(lib().gemm_f16_splitk_bt(_ptr(A), _ptr(Bt), _ptr(C), out, M, N, K, ws, nbytes, _stream_handle(stream)),
           "gemm_f16_splitk_bt")
    return C


def gemm_fp8_exact(A, fmt_a, B, fmt_b, sA, sB, C, sOut=None, stream=None, out_fmt=None):
    """gemm_fp8_fmt with exact products and FP32 additions throughout (the
    codes widened to FP16 on the FP16 matrix cores, or the FP32-FMA decode
    kernels)."""
    A, B = _u8(A, fmt_a), _u8(B, fmt_b)
    out = _out_dtype(C, out_fmt)
    Cv = _u8(C) if out in (OUT_E4M3, OUT_E5M2) else C
    M, N, K = _dims(A, B, Cv)
    _check(lib().gemm_fp8_exact(_ptr(A), int(fmt_a), _ptr(B), int(fmt_b), _ptr(sA), _ptr(sB), _ptr(sOut), _ptr(Cv),
                                out, M, N, K, _stream_handle(stream)), "gemm_fp8_exact")
    return C


def gemm_fp8_exact_bt(A, fmt_a, Bt, fmt_b, sA, sB, C, sOut=None, stream=None, out_fmt=None):
    """gemm_fp8_exact with B given K-major as Bt[N,K]."""
    A, Bt = _u8(A, fmt_a), _u8(Bt, fmt_b)
    out = _out_dtype(C, out_fmt)
    Cv = _u8(C) if out in (OUT_E4M3, OUT_E5M2) else C
    M, N, K = _dims_bt(A, Bt, Cv)
    _check(lib().gemm_fp8_exact_bt(_ptr(A), int(fmt_a), _ptr(Bt), int(fmt_b), _ptr(sA), _ptr(sB), _ptr(sOut),
                                   _ptr(Cv), out, M, N, K, _stream_handle(stream)), "gemm_fp8_exact_bt")
    return C


def select_config_exact(out_dtype: int, M: int, N: int, K: int, fmt_a: int = 0, fmt_b: int = 0,
                        b_kmajor: int = 0) -> str:
    """The configuration gemm_fp8_exact (or, with b_kmajor, gemm_fp8_exact_bt) would launch."""
    buf = ctypes.create_string_buffer(128)
    _check(lib().gemm_select_config_exact(out_dtype, M, N, K, int(fmt_a), int(fmt_b), int(b_kmajor), buf, len(buf)),
           "gemm_select_config_exact")
    return buf.value.decode()


def amax_quantize_fp8_pair(xa, xb, fmt=FMT_E4M3, pow2=False, amax=None, scale=None, qa=None, qb=None,
                           workspace=None, stream=None):
    """amax, scale and FP8 codes of two float32 tensors in two launches:
    returns (amax[2], scale[2], qa, qb), bit-identical to amax_scale_f32 and
    quantize_fp8_fmt on each. xb may be None (then amax and scale have one
    element and qb is None)."""
    torch = _torch()
    for name, x in (("xa", xa), ("xb", xb)):
        if x is not None and x.dtype != torch.float32:
            raise ValueError(f"{name} must be float32")
    dev = xa.device
    two = xb is not None
    if amax is None:
        amax = torch.empty(2 if two else 1, dtype=torch.float32, device=dev)
    if scale is None:
        scale = torch.empty(2 if two else 1, dtype=torch.float32, device=dev)
    if qa is None:
        qa = torch.empty(xa.shape, dtype=torch.uint8, device=dev)
    if two and qb is None:
        qb = torch.empty(xb.shape, dtype=torch.uint8, device=dev)
    qav = _u8(qa, fmt)
    qbv = _u8(qb, fmt) if two else None
    if qav.numel() != xa.numel() or (two and qbv.numel() != xb.numel()):
        raise ValueError("q must have as many elements as its x")
    if amax.numel() < (2 if two else 1) or scale.numel() < (2 if two else 1):
        raise ValueError("amax and scale need one element per tensor")
    if workspace is None:
        workspace = torch.empty(int(lib().amax_quantize_fp8_pair_workspace_size()), dtype=torch.uint8, device=dev)
    _check(lib().amax_quantize_fp8_pair(_ptr(xa), xa.numel(), _ptr(xb) if two else None, xb.numel() if two else 0,
                                        int(fmt), 1 if pow2 else 0, _ptr(amax), _ptr(scale), _ptr(qav),
                                        _ptr(qbv) if two else None, _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream_handle(stream)),
           "amax_quantize_fp8_pair")
    return amax, scale, qa, qb


def amax_quantize_fp8_pair_bt(xa, xb, fmt=FMT_E4M3, pow2=False, amax=None, scale=None, qa=None, qbt=None,
                              workspace=None, stream=None):
    """amax_quantize_fp8_pair for a row-major float32 xb[K, N] whose codes are
    written K-major: returns (amax[2], scale[2], qa, qbt) with qbt[N, K] the
    transpose of amax_quantize_fp8_pair's qb, for the gemm_*_bt calls."""
    torch = _torch()
    for name, x in (("xa", xa), ("xb", xb)):
        if x.dtype != torch.float32:
            raise ValueError(f"{name} must be float32")
    if xb.dim() != 2 or not xb.is_contiguous():
        raise ValueError("xb must be a contiguous [K, N] matrix")
    K, N = xb.shape
    dev = xa.device
    if amax is None:
        amax = torch.empty(2, dtype=torch.float32, device=dev)
    if scale is None:
        scale = torch.empty(2, dtype=torch.float32, device=dev)
    if qa is None:
        qa = torch.empty(xa.shape, dtype=torch.uint8, device=dev)
    if qbt is None:
        qbt = torch.empty((N, K), dtype=torch.uint8, device=dev)
    qav, qbv = _u8(qa, fmt), _u8(qbt, fmt)
    if qav.numel() != xa.numel() or qbv.numel() != xb.numel():
        raise ValueError("q must have as many elements as its x")
    if amax.numel() < 2 or scale.numel() < 2:
        raise ValueError("amax and scale need one element per tensor")
    if workspace is None:
        workspace = torch.empty(int(lib().amax_quantize_fp8_pair_workspace_size()), dtype=torch.uint8, device=dev)
    _check(lib().amax_quantize_fp8_pair_bt(_ptr(xa), xa.numel(), _ptr(xb), K, N, int(fmt), 1 if pow2 else 0,
                                           _ptr(amax), _ptr(scale), _ptr(qav), _ptr(qbv), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream_handle(stream)),
           "amax_quantize_fp8_pair_bt")
    return amax, scale, qa, qbt


# ------------------------------------ products whose weight depends on the row

def _need(t, dtype, shape, what):
    """Checks an argument's type and shape (an int in place of the shape: that many dimensions, of any size)."""
    if t.dtype is dtype and (t.dim() if shape.__class__ is int else t.shape) == shape:
        return
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, not {t.dtype}")
    raise ValueError(f"{what} must have {shape} dimensions, not shape {tuple(t.shape)}" if isinstance(shape, int) else
                     f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _arg(t, dtype, shape, what):
    """_need and _ptr in one."""
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():   # the common case
        return t.data_ptr()
    _need(t, dtype, shape, what)
    return _ptr(t)


def _new(shape, dtype, device, stream, zero=False):
    """An output or workspace of a call on `stream`: allocated (and cleared) on that stream, so that neither memory
    another stream is still using nor a clear on another stream meets the call."""
    torch = _torch()
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _grouped_dims(A, B, offsets, C, bt):
    if A.dim() != 2 or B.dim() != 3 or C.dim() != 2:
        raise ValueError("A and C must be 2-D and B 3-D, one weight per group")
    rows, K = A.shape
    groups = B.shape[0]
    N, K2 = (B.shape[1], B.shape[2]) if bt else (B.shape[2], B.shape[1])
    if K2 != K or tuple(C.shape) != (rows, N):
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    _need(offsets, _torch().int32, (groups + 1,), "offsets")
    return rows, N, K, groups


def _grouped_f16(name, A, B, offsets, C, bt, stream):
    torch = _torch()
    if A.dtype != torch.float16 or B.dtype != torch.float16:
        raise ValueError(f"{name} takes float16 operands")
    rows, N, K, groups = _grouped_dims(A, B, offsets, C, bt)
    _check(getattr(lib(), name)(_ptr(A), _ptr(B), _ptr(offsets), _ptr(C), _out_dtype(C), rows, N, K, groups,
                                _stream_handle(stream)), name)
    return C


def gemm_f16_grouped(A, B, offsets, C, stream=None):
    """C[r] = A[r] @ B[g] for the rows offsets[g] <= r < offsets[g + 1]; float16 A[rows, K] and B[groups, K, N],
    int32 offsets[groups + 1] on the device; C float32 or float16 [rows, N], zeros in rows of no group."""
    return _grouped_f16("gemm_f16_grouped", A, B, offsets, C, False, stream)


def gemm_f16_grouped_bt(A, Bt, offsets, C, stream=None):
    """gemm_f16_grouped with K-major weights Bt[groups, N, K]: C[r] = A[r] @ Bt[g].T."""
    return _grouped_f16("gemm_f16_grouped_bt", A, Bt, offsets, C, True, stream)


def _grouped_fp8(name, A, fmt_a, B, fmt_b, offsets, sA, sB, C, sOut, stream, out_fmt, bt, channel):
    torch = _torch()
    A, B = _u8(A, fmt_a), _u8(B, fmt_b)
    out = _out_dtype(C, out_fmt)
    Cv = _u8(C) if out in (OUT_E4M3, OUT_E5M2) else C
    rows, N, K, groups = _grouped_dims(A, B, offsets, Cv, bt)
    for what, s, n in (("sA", sA, rows if channel else 1), ("sB", sB, groups * N if channel else groups)):
        if s.dtype != torch.float32 or s.numel() != n:
            raise ValueError(f"{what} must hold {n} float32 scales")
    _check(getattr(lib(), name)(_ptr(A), int(fmt_a), _ptr(B), int(fmt_b), _ptr(offsets), _ptr(sA), _ptr(sB),
                                _ptr(sOut), _ptr(Cv), out, rows, N, K, groups, _stream_handle(stream)), name)
    return C


def gemm_fp8_grouped(A, fmt_a, B, fmt_b, offsets, sA, sB, C, sOut=None, stream=None, out_fmt=None):
    """gemm_f16_grouped for FP8 codes A[rows, K] and B[groups, K, N]: C[r] = (sA*A[r]) @ (sB[g]*B[g]), sA one
    float32 scale, sB one per group; C float32, float16 or 8-bit codes (with sOut)."""
    return _grouped_fp8("gemm_fp8_grouped", A, fmt_a, B, fmt_b, offsets, sA, sB, C, sOut, stream, out_fmt, False,
                        False)


def gemm_fp8_grouped_bt(A, fmt_a, Bt, fmt_b, offsets, sA, sB, C, sOut=None, stream=None, out_fmt=None):
    """gemm_fp8_grouped with K-major weights Bt[groups, N, K]."""
    return _grouped_fp8("gemm_fp8_grouped_bt", A, fmt_a, Bt, fmt_b, offsets, sA, sB, C, sOut, stream, out_fmt, True,
                        False)


def gemm_fp8_grouped_channel(A, fmt_a, B, fmt_b, offsets, sA, sB, C, sOut=None, stream=None, out_fmt=None):
    """gemm_fp8_grouped with a scale per row of A (sA[rows]) and per output column of each weight (sB[groups, N])."""
    return _grouped_fp8("gemm_fp8_grouped_channel", A, fmt_a, B, fmt_b, offsets, sA, sB, C, sOut, stream, out_fmt,
                        False, True)


def gemm_fp8_grouped_channel_bt(A, fmt_a, Bt, fmt_b, offsets, sA, sB, C, sOut=None, stream=None, out_fmt=None):
    """gemm_fp8_grouped_channel with K-major weights Bt[groups, N, K]."""
    return _grouped_fp8("gemm_fp8_grouped_channel_bt", A, fmt_a, Bt, fmt_b, offsets, sA, sB, C, sOut, stream, out_fmt,
                        True, True)


def gemm_f16_grouped_wgrad(A, B, offsets, C, stream=None):
    """C[g] = A[rows of g].T @ B[rows of g] for float16 A[rows, M], B[rows, N]; C float32 or float16 [groups, M, N],
    zeros for an empty group."""
    torch = _torch()
    if A.dtype != torch.float16 or B.dtype != torch.float16:
        raise ValueError("gemm_f16_grouped_wgrad takes float16 operands")
    if A.dim() != 2 or B.dim() != 2 or C.dim() != 3 or A.shape[0] != B.shape[0]:
        raise ValueError("A[rows, M], B[rows, N] and C[groups, M, N] are needed")
    rows, M, N, groups = A.shape[0], A.shape[1], B.shape[1], C.shape[0]
    if tuple(C.shape) != (groups, M, N):
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    _need(offsets, torch.int32, (groups + 1,), "offsets")
    _check(lib().gemm_f16_grouped_wgrad(_ptr(A), _ptr(B), _ptr(offsets), _ptr(C), _out_dtype(C), rows, M, N, groups,
                                        _stream_handle(stream)), "gemm_f16_grouped_wgrad")
    return C


def select_config_grouped(kind: int, out_dtype: int, rows: int, N: int, K: int, groups: int, fmt_a: int = 0,
                          fmt_b: int = 0, b_kmajor: int = 0) -> str:
    """The kernel that the grouped products (kind KIND_F16 or KIND_FP8; K-major weights with b_kmajor) would launch for
    16-byte aligned operands."""
    buf = ctypes.create_string_buffer(128)
    _check(lib().gemm_select_config_grouped(kind, out_dtype, rows, N, K, groups, int(fmt_a), int(fmt_b), int(b_kmajor),
                                            buf, len(buf)), "gemm_select_config_grouped")
    return buf.value.decode()


def select_config_wgrad(out_dtype: int, rows: int, M: int, N: int, groups: int) -> str:
    """The kernel that gemm_f16_grouped_wgrad would launch for 16-byte aligned operands."""
    buf = ctypes.create_string_buffer(128)
    _check(lib().gemm_select_config_wgrad(out_dtype, rows, M, N, groups, buf, len(buf)), "gemm_select_config_wgrad")
    return buf.value.decode()


def select_config_lora(kind: int, out_dtype: int, rows: int, N: int, K: int, rank: int, adapters: int, fmt_a: int = 0,
                       fmt_b: int = 0) -> str:
    """The kernel of the product that gemm_f16_lora_bt (KIND_F16) or gemm_fp8_lora_bt (KIND_FP8) would launch for
    16-byte aligned operands."""
    buf = ctypes.create_string_buffer(128)
    _check(lib().gemm_select_config_lora(kind, out_dtype, rows, N, K, rank, adapters, int(fmt_a), int(fmt_b), buf,
                                         len(buf)), "gemm_select_config_lora")
    return buf.value.decode()


def lora_workspace_size(rows: int, rank: int) -> int:
    n = int(lib().gemm_lora_workspace_size(rows, rank))
    _check(n if n < 0 else 0, "gemm_lora_workspace_size")
    return n


def _lora_dims(X, N, LA, LB, adapter, lscale, workspace, stream):
    torch = _torch()
    rows, K = X.shape
    if LA.dim() != 3 or LB.dim() != 3:
        raise ValueError("LA[adapters, rank, K] and LB[adapters, N, rank] are needed")
    adapters, rank = LA.shape[0], LA.shape[1]
    args = (_arg(LA, torch.float16, (adapters, rank, K), "LA"), _arg(LB, torch.float16, (adapters, N, rank), "LB"),
            _arg(adapter, torch.int32, (rows,), "adapter"), _arg(lscale, torch.float32, (adapters,), "lscale"))
    if workspace is None:
        workspace = _new(lora_workspace_size(rows, rank), torch.uint8, X.device, stream)
    return rows, K, rank, adapters, args, workspace


def gemm_f16_lora_bt(A, Bt, LA, LB, adapter, lscale, C, workspace=None, stream=None):
    """C[r] = A[r] @ Bt.T + lscale[a] * (A[r] @ LA[a].T) @ LB[a].T with a = adapter[r] (int32, -1: none); float16
    A[rows, K], Bt[N, K], LA[adapters, rank, K], LB[adapters, N, rank], float32 lscale[adapters]; C float32 or
    float16 [rows, N]. workspace: lora_workspace_size(rows, rank) bytes, allocated when None."""
    torch = _torch()
    if A.dtype != torch.float16 or Bt.dtype != torch.float16:
        raise ValueError("gemm_f16_lora_bt takes float16 operands")
    M, N, K = _dims_bt(A, Bt, C)
    rows, K, rank, adapters, low, ws = _lora_dims(A, N, LA, LB, adapter, lscale, workspace, stream)
    _check(lib().gemm_f16_lora_bt(_ptr(A), _ptr(Bt), *low, _ptr(C), _out_dtype(C), rows, N, K, rank,
                                  adapters, *_ws_args(ws), _stream_handle(stream)), "gemm_f16_lora_bt")
    return C


def gemm_fp8_lora_bt(A, fmt_a, Bt, fmt_b, sA, sB, X, LA, LB, adapter, lscale, C, workspace=None, stream=None):
    """gemm_f16_lora_bt with the shared product in FP8: codes A[rows, K] and Bt[N, K] with float32 scales sA[rows]
    and sB[N], and the float16 activations X[rows, K] that the adapters multiply."""
    torch = _torch()
    A, Bt = _u8(A, fmt_a), _u8(Bt, fmt_b)
    M, N, K = _dims_bt(A, Bt, C)
    _need(sA, torch.float32, (M,), "sA")
    _need(sB, torch.float32, (N,), "sB")
    _need(X, torch.float16, (M, K), "X")
    rows, K, rank, adapters, low, ws = _lora_dims(X, N, LA, LB, adapter, lscale, workspace, stream)
    _check(lib().gemm_fp8_lora_bt(_ptr(A), int(fmt_a), _ptr(Bt), int(fmt_b), _ptr(sA), _ptr(sB), _ptr(X), *low, _ptr(C),
                                  _out_dtype(C), rows, N, K, rank, adapters, *_ws_args(ws), _stream_handle(stream)), "gemm_fp8_lora_bt")
    return C


# -------------------------------------------------------------- expert routing

def moe_route_workspace_size(tokens: int, experts: int) -> int:
    n = int(lib().moe_route_workspace_size(tokens, experts))
    _check(n if n < 0 else 0, "moe_route_workspace_size")
    return n


def moe_route_f32(logits, topk, renorm=True, expert=None, weight=None, offsets=None, row=None, token=None,
                  workspace=None, stream=None):
    """The topk experts of each token and the order of the rows by expert, from float32 logits[tokens, experts]:
    (expert[tokens, topk] int32, weight[tokens, topk] float32, offsets[experts + 1], row[tokens, topk],
    token[tokens * topk]). Equal logits go to the lower index; -inf and NaN are never chosen (expert and row -1,
    weight 0). renorm: weights sum to 1 over the chosen experts, else they are the softmax over all."""
    torch = _torch()
    _need(logits, torch.float32, 2, "logits")
    T, E = logits.shape
    topk = int(topk)
    dev = logits.device
    if topk < 1 or topk > E:
        raise ValueError(f"topk must be between 1 and the {E} experts, not {topk}")

    i32, f32 = torch.int32, torch.float32
    if expert is None:
        expert = _new((T, topk), i32, dev, stream)
    if weight is None:
        weight = _new((T, topk), f32, dev, stream)
    if offsets is None:
        offsets = _new((E + 1,), i32, dev, stream)
    if row is None:
        row = _new((T, topk), i32, dev, stream)
    if token is None:
        token = _new((T * topk,), i32, dev, stream)
    per = (T, topk)
    outs = (_arg(expert, i32, per, "expert"), _arg(weight, f32, per, "weight"), _arg(offsets, i32, (E + 1,), "offsets"),
            _arg(row, i32, per, "row"), _arg(token, i32, (T * topk,), "token"))
    if workspace is None:
        n = moe_route_workspace_size(T, E)
        workspace = _new(n, torch.uint8, dev, stream) if n else None
    _check(lib().moe_route_f32(_ptr(logits), T, E, topk, 1 if renorm else 0, *outs, *_ws_args(workspace),
                               _stream_handle(stream)), "moe_route_f32")
    return expert, weight, offsets, row, token


def moe_route_backward_f32(logits, expert, weight, dweight, renorm=True, dlogits=None, stream=None):
    """dlogits[tokens, experts] of moe_route_f32's weights, from dweight[tokens, topk]."""
    torch = _torch()
    _need(logits, torch.float32, 2, "logits")
    T, E = logits.shape
    _need(expert, torch.int32, 2, "expert")
    K = expert.shape[1]
    _need(expert, torch.int32, (T, K), "expert")
    _need(weight, torch.float32, (T, K), "weight")
    _need(dweight, torch.float32, (T, K), "dweight")
    if dlogits is None:
        dlogits = _new((T, E), torch.float32, logits.device, stream)
    _need(dlogits, torch.float32, (T, E), "dlogits")
    _check(lib().moe_route_backward_f32(_ptr(logits), _ptr(expert), _ptr(weight), _ptr(dweight), T, E, K,
                                        1 if renorm else 0, _ptr(dlogits), _stream_handle(stream)),
           "moe_route_backward_f32")
    return dlogits


def moe_gather(x, token, y=None, stream=None):
    """y[r] = x[token[r]] for x[tokens, width] of any 1-, 2- or 4-byte type and int32 token[rows]; zeros where
    token[r] is outside [0, tokens)."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("x must be [tokens, width]")
    _need(token, torch.int32, 1, "token")
    rows = token.shape[0]
    if y is None:
        y = _new((rows, x.shape[1]), x.dtype, x.device, stream)
    tokens, width = x.shape
    py = _arg(y, x.dtype, (rows, width), "y")
    _check(lib().moe_gather(_ptr(x), _ptr(token), py, tokens, rows, width, x.element_size(),
                            _stream_handle(stream)), "moe_gather")
    return y


def _float_dtype(t, what):
    torch = _torch()
    if t.dtype == torch.float32:
        return OUT_F32
    if t.dtype == torch.float16:
        return OUT_F16
    raise ValueError(f"{what} must be float32 or float16, not {t.dtype}")


def moe_combine(z, row, weight, y=None, stream=None):
    """y[t] = sum_j weight[t, j] * z[row[t, j]] over the j with a row (int32 row[tokens, topk], -1: none), summed in
    float32; z[rows, width] and y[tokens, width] float32 or float16 (y as z when None). weight None: all 1, the
    gradient of moe_gather."""
    torch = _torch()
    zt = _float_dtype(z, "z")
    if z.dim() != 2:
        raise ValueError("z must be [rows, width]")
    _need(row, torch.int32, 2, "row")
    T, K = row.shape
    rows, width = z.shape
    pw = None if weight is None else _arg(weight, torch.float32, (T, K), "weight")
    if y is None:
        y = _new((T, width), z.dtype, z.device, stream)
    yt = _float_dtype(y, "y")
    py = _arg(y, y.dtype, (T, width), "y")
    _check(lib().moe_combine(_ptr(z), zt, _ptr(row), pw, py, yt, T, K, rows, width,
                             _stream_handle(stream)), "moe_combine")
    return y


def moe_combine_backward(dy, z, row, weight, dZ=None, dweight=None, stream=None):
    """(dZ, dweight) of moe_combine: dZ[row[t, j]] = weight[t, j] * dy[t], dweight[t, j] = <z[row[t, j]], dy[t]>.
    dy, z and dZ are of one type (float32 or float16). Rows that no (t, j) names are not written; dZ=None allocates
    zeros."""
    torch = _torch()
    dt = _float_dtype(z, "z")
    _need(row, torch.int32, 2, "row")
    T, K = row.shape
    pw = _arg(weight, torch.float32, (T, K), "weight")
    _need(z, z.dtype, 2, "z")
    rows, width = z.shape
    pdy = _arg(dy, z.dtype, (T, width), "dy")
    if dZ is None:
        dZ = _new((rows, width), z.dtype, z.device, stream, zero=True)
    if dweight is None:
        dweight = _new((T, K), torch.float32, z.device, stream)
    pdz, pdw = _arg(dZ, z.dtype, (rows, width), "dZ"), _arg(dweight, torch.float32, (T, K), "dweight")
    _check(lib().moe_combine_backward(pdy, _ptr(z), dt, _ptr(row), pw, pdz, pdw, T, K, rows, width,
                                      _stream_handle(stream)), "moe_combine_backward")
    return dZ, dweight


# ------------------------------------------- a dense layer around its products

def _codes_ptr(t, fmt=None):
    """_ptr(_u8(t, fmt)) without making the view (1 us of a call)."""
    torch = _torch()
    have = FMT_E4M3 if t.dtype is torch.float8_e4m3fn else (FMT_E5M2 if t.dtype is torch.float8_e5m2 else None)
    if t.dtype is torch.uint8 or (have is not None and (fmt is None or int(fmt) == have)):
        return _ptr(t)
    return _ptr(_u8(t, fmt))


def _mx_codes(q, scale, fmt, what):
    """Pointers of 8-bit values q[rows, cols] and their scales [rows, ceil(cols / 32)]."""
    torch = _torch()
    if q.dim() != 2:
        raise ValueError(f"{what} must be [rows, cols]")
    if scale is None:
        raise ValueError(f"{what} holds 8-bit values: their scales are needed")
    if scale.dtype != torch.uint8:
        if scale.dtype != getattr(torch, "float8_e8m0fnu", None):
            raise ValueError(f"{what}'s scales must be uint8 or float8_e8m0fnu, not {scale.dtype}")
        scale = scale.view(torch.uint8)
    shape = (q.shape[0], (q.shape[1] + 31) // 32)
    return _codes_ptr(q, fmt), _arg(scale, torch.uint8, shape, f"{what}'s scales")


def _held(t, scale, fmt, shape, what):
    """(pointer, scales' pointer, type) of a matrix of float32, float16 or 8-bit values."""
    torch = _torch()
    dt = _out_dtype(t, fmt)
    if dt in (OUT_E4M3, OUT_E5M2):
        if t.shape != shape:
            raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
        return (*_mx_codes(t, scale, None, what), dt)
    return _arg(t, t.dtype, shape, what), None, dt


def _opt(t, dtype, shape, what):
    return None if t is None else _arg(t, dtype, shape, what)


def rms_norm(x, weight, y, eps=1e-5, residual=None, h=None, scale=None, rstd=None, pow2=False, out_fmt=None, stream=None):
    """y = h * weight / sqrt(mean(h^2) + eps) row by row, h = x + residual rounded to x's type (written to h when given).
    x[rows, width], residual and h float32 or float16, weight[width] float32; y float32, float16 or FP8 codes with
    scale[rows] float32 (max|y| / fmax, or its power of two). rstd[rows] float32, written when given, is what the
    backward pass takes."""
    torch = _torch()
    dt = _float_dtype(x, "x")
    _need(x, x.dtype, 2, "x")
    rows, width = shape = x.shape
    yt = _out_dtype(y, out_fmt)
    if y.shape != shape:
        raise ValueError(f"y must have shape {tuple(shape)}, not {tuple(y.shape)}")
    codes = yt in (OUT_E4M3, OUT_E5M2)
    if codes and scale is None:
        raise ValueError("FP8 output needs scale[rows]")
    f32 = torch.float32
    _check(lib().rms_norm(_ptr(x), _opt(residual, x.dtype, shape, "residual"), dt, _arg(weight, f32, (width,), "weight"),
                          eps, _opt(h, x.dtype, shape, "h"), _ptr(y), yt,
                          _opt(scale if codes else None, f32, (rows,), "scale"), 1 if pow2 else 0,
                          _opt(rstd, f32, (rows,), "rstd"), rows, width, _stream_handle(stream)), "rms_norm")
    return y


def rms_norm_backward_workspace_size(rows: int, width: int) -> int:
    n = int(lib().rms_norm_backward_workspace_size(rows, width))
    _check(n if n < 0 else 0, "rms_norm_backward_workspace_size")
    return n


def rms_norm_backward(dy, h, weight, rstd, dx=None, dweight=None, dh=None, hscale=None, h_fmt=None, workspace=None,
                      stream=None):
    """(dx, dweight) of rms_norm. dy, dh (the gradient of h itself, added to dx) and dx are of one type, float32 or
    float16; h as rms_norm wrote it, or 8-bit values of it with hscale; rstd[rows] as rms_norm wrote it. dweight is
    computed when given (None otherwise; the workspace is then needed for rows of more than 16384 values only)."""
    torch = _torch()
    dt = _float_dtype(dy, "dy")
    _need(dy, dy.dtype, 2, "dy")
    rows, width = shape = dy.shape
    f32 = torch.float32
    if dx is None:
        dx = _new(shape, dy.dtype, dy.device, stream)
    ph, ps, ht = _held(h, hscale, h_fmt, shape, "h")
    if workspace is None:
        # (without dweight the long rows' own words alone)
        n = rms_norm_backward_workspace_size(rows, width) if dweight is not None else (4 * rows if width > 16384 else 0)
        workspace = _new(n, torch.uint8, dy.device, stream) if n else None
    _check(lib().rms_norm_backward(_ptr(dy), _opt(dh, dy.dtype, shape, "dh"), dt, ph, ps, ht,
                                   _arg(weight, f32, (width,), "weight"), _arg(rstd, f32, (rows,), "rstd"),
                                   _arg(dx, dy.dtype, shape, "dx"), _opt(dweight, f32, (width,), "dweight"), rows,
                                   width, *_ws_args(workspace), _stream_handle(stream)), "rms_norm_backward")
    return dx, dweight


def _epilogue(C, bias, residual, Z, Zscale, z_fmt):
    """Pointers and types of the epilogue's operands for C[M, N]."""
    torch = _torch()
    shape = C.shape
    pb = _opt(bias, torch.float32, (shape[1],), "bias")
    pr, rt = None, 0
    if residual is not None:
        rt = _float_dtype(residual, "residual")
        pr = _arg(residual, residual.dtype, shape, "residual")
    pz, ps, zt = (None, None, 0) if Z is None else _held(Z, Zscale, z_fmt, shape, "Z")
    return pb, pr, rt, pz, ps, zt


def _bias_act_f16(name, A, B, C, bias, act, residual, Z, Zscale, z_fmt, stream, bt):
    torch = _torch()
    if A.dtype != torch.float16 or B.dtype != torch.float16:
        raise ValueError(f"{name} takes float16 operands")
    M, N, K = _dims_bt(A, B, C) if bt else _dims(A, B, C)
    pb, pr, rt, pz, ps, zt = _epilogue(C, bias, residual, Z, Zscale, z_fmt)
    _check(getattr(lib(), name)(_ptr(A), _ptr(B), pb, pr, rt, _ptr(C), _out_dtype(C), int(act), pz, ps, zt, M, N, K,
                                _stream_handle(stream)), name)
    return C


def gemm_f16_bias_act(A, B, C, bias=None, act=ACT_NONE, residual=None, Z=None, Zscale=None, z_fmt=None, stream=None):
    """C = act(A @ B + bias) + residual for float16 A[M, K] and B[K, N]; C and residual[M, N] float32 or float16,
    bias[N] float32. Z, when given, takes A @ B + bias: float32, float16, or 8-bit values with Zscale."""
    return _bias_act_f16("gemm_f16_bias_act", A, B, C, bias, act, residual, Z, Zscale, z_fmt, stream, False)


def gemm_f16_bias_act_bt(A, Bt, C, bias=None, act=ACT_NONE, residual=None, Z=None, Zscale=None, z_fmt=None,
                         stream=None):
    """gemm_f16_bias_act with a K-major weight Bt[N, K]."""
    return _bias_act_f16("gemm_f16_bias_act_bt", A, Bt, C, bias, act, residual, Z, Zscale, z_fmt, stream, True)


def _bias_act_fp8(name, A, fmt_a, B, fmt_b, sA, sB, C, bias, act, residual, Z, Zscale, channel, sOut, out_fmt, z_fmt,
                  stream, bt):
    torch = _torch()
    pa, pw = _codes_ptr(A, fmt_a), _codes_ptr(B, fmt_b)
    out = _out_dtype(C, out_fmt)
    codes = out in (OUT_E4M3, OUT_E5M2)
    M, N, K = _dims_bt(A, B, C) if bt else _dims(A, B, C)
    for what, s, n in (("sA", sA, M if channel else 1), ("sB", sB, N if channel else 1),
                       ("sOut", sOut if codes else None, 1)):
        if s is not None and (s.dtype != torch.float32 or s.numel() != n):
            raise ValueError(f"{what} must hold {n} float32 scales")
    pb, pr, rt, pz, ps, zt = _epilogue(C, bias, residual, Z, Zscale, z_fmt)
    _check(getattr(lib(), name)(pa, int(fmt_a), pw, int(fmt_b), _ptr(sA), _ptr(sB), 1 if channel else 0,
                                _ptr(sOut) if codes else None, pb, pr, rt, _ptr(C), out, int(act), pz, ps, zt, M, N,
                                K, _stream_handle(stream)), name)
    return C


def gemm_fp8_bias_act(A, fmt_a, B, fmt_b, sA, sB, C, bias=None, act=ACT_NONE, residual=None, Z=None, Zscale=None,
                      channel=False, sOut=None, out_fmt=None, z_fmt=None, stream=None):
    """C = act((sA*A) @ (sB*B) + bias) + residual for FP8 codes; sA and sB one float32 scale each, or with channel
    sA[M] and sB[N]. C float32, float16 or FP8 codes (divided by sOut); the rest as gemm_f16_bias_act."""
    return _bias_act_fp8("gemm_fp8_bias_act", A, fmt_a, B, fmt_b, sA, sB, C, bias, act, residual, Z, Zscale, channel,
                         sOut, out_fmt, z_fmt, stream, False)


def gemm_fp8_bias_act_bt(A, fmt_a, Bt, fmt_b, sA, sB, C, bias=None, act=ACT_NONE, residual=None, Z=None, Zscale=None,
                         channel=False, sOut=None, out_fmt=None, z_fmt=None, stream=None):
    """gemm_fp8_bias_act with a K-major weight Bt[N, K]."""
    return _bias_act_fp8("gemm_fp8_bias_act_bt", A, fmt_a, Bt, fmt_b, sA, sB, C, bias, act, residual, Z, Zscale,
                         channel, sOut, out_fmt, z_fmt, stream, True)


def select_config_bias_act(kind: int, out_dtype: int, M: int, N: int, K: int, fmt_a: int = 0, fmt_b: int = 0,
                           b_kmajor: int = 0, z_dtype: int = -1) -> str:
    """The kernel that the products with bias, activation and residual would launch for 16-byte aligned operands."""
    buf = ctypes.create_string_buffer(128)
    _check(lib().gemm_select_config_bias_act(kind, out_dtype, M, N, K, int(fmt_a), int(fmt_b), int(b_kmajor),
                                             int(z_dtype), buf, len(buf)), "gemm_select_config_bias_act")
    return buf.value.decode()


def bias_act_backward_workspace_size(rows: int, cols: int) -> int:
    n = int(lib().bias_act_backward_workspace_size(rows, cols))
    _check(n if n < 0 else 0, "bias_act_backward_workspace_size")
    return n


def bias_act_backward(dy, Z, act, dZ=None, dbias=None, Zscale=None, z_fmt=None, workspace=None, stream=None):
    """(dZ, dbias) of the epilogue act(z) + residual, z = product + bias: dZ = dy * act'(z), dbias its column sums.
    dy and dZ are of one type, float32 or float16; Z float32, float16 or 8-bit values with Zscale (None for ACT_NONE).
    dbias is computed when given (None otherwise)."""
    torch = _torch()
    dt = _float_dtype(dy, "dy")
    _need(dy, dy.dtype, 2, "dy")
    rows, cols = shape = dy.shape
    if dZ is None:
        dZ = _new(shape, dy.dtype, dy.device, stream)
    pz, ps, zt = (None, None, 0) if Z is None else _held(Z, Zscale, z_fmt, shape, "Z")
    if workspace is None and dbias is not None:
        n = bias_act_backward_workspace_size(rows, cols)
        workspace = _new(n, torch.uint8, dy.device, stream) if n else None
    _check(lib().bias_act_backward(_ptr(dy), dt, pz, ps, zt, int(act), _arg(dZ, dy.dtype, shape, "dZ"),
                                   _opt(dbias, torch.float32, (cols,), "dbias"), rows, cols, *_ws_args(workspace),
                                   _stream_handle(stream)), "bias_act_backward")
    return dZ, dbias


def quantize_mx_fp8(x, fmt=FMT_E4M3, q=None, scale=None, stream=None):
    """8-bit values of float32 or float16 x[rows, cols]: (codes[rows, cols], scale[rows, ceil(cols / 32)]), a power of
    two 2^(scale - 127) per 32 values of a row. What the codes of float16 x stand for are float16 numbers; float32 x may
    lie past their range, which gemm_mx_wgrad and dequantize_mx_fp8 into float16 read as infinities or zeros."""
    torch = _torch()
    dt = _float_dtype(x, "x")
    _need(x, x.dtype, 2, "x")
    rows, cols = x.shape
    if q is None:
        q = _new((rows, cols), torch.uint8, x.device, stream)
    if scale is None:
        scale = _new((rows, (cols + 31) // 32), torch.uint8, x.device, stream)
    if q.shape != x.shape:
        raise ValueError(f"q must have shape {tuple(x.shape)}, not {tuple(q.shape)}")
    pq, ps = _mx_codes(q, scale, fmt, "q")
    _check(lib().quantize_mx_fp8(_ptr(x), dt, rows, cols, int(fmt), pq, ps, _stream_handle(stream)), "quantize_mx_fp8")
    return q, scale


def dequantize_mx_fp8(q, scale, fmt, y, stream=None):
    """What 8-bit values stand for, into float32 or float16 y[rows, cols]."""
    dt = _float_dtype(y, "y")
    pq, ps = _mx_codes(q, scale, fmt, "q")
    rows, cols = q.shape
    _check(lib().dequantize_mx_fp8(pq, ps, int(fmt), rows, cols, _arg(y, y.dtype, q.shape, "y"), dt,
                                   _stream_handle(stream)), "dequantize_mx_fp8")
    return y


def gemm_mx_wgrad(q, scale, fmt, B, C, offsets=None, q_second=False, stream=None):
    """X.T @ B for 8-bit values X (q[rows, M], scale; multiplied as float16 numbers, past 65504 infinite, below 2^-25
    zero) and float16 B[rows, N], into float32 or float16 C[M, N]; with q_second B.T @ X into C[N, M]. With offsets[groups + 1] one product per group of rows, C[groups, ...]."""
    torch = _torch()
    pq, ps = _mx_codes(q, scale, fmt, "q")
    rows, M = q.shape
    _need(B, torch.float16, 2, "B")
    N = B.shape[1]
    if B.shape[0] != rows:
        raise ValueError(f"q and B must have the same rows, not {rows} and {B.shape[0]}")
    one = (N, M) if q_second else (M, N)
    groups = 1
    if offsets is not None:
        _need(offsets, torch.int32, 1, "offsets")
        groups = offsets.shape[0] - 1
        one = (groups, *one)
    if groups < 0:
        raise ValueError("offsets must hold groups + 1 values")
    ct = _float_dtype(C, "C")
    _check(lib().gemm_mx_wgrad(pq, ps, int(fmt), _ptr(B), _ptr(offsets), _arg(C, C.dtype, one, "C"), ct, rows, M, N,
                               groups, 1 if q_second else 0, _stream_handle(stream)), "gemm_mx_wgrad")
    return C


def select_config_mx_wgrad(out_dtype: int, rows: int, M: int, N: int, groups: int = 1, q_second: bool = False) -> str:
    """The kernel that gemm_mx_wgrad would launch for 16-byte aligned operands."""
    buf = ctypes.create_string_buffer(128)
    _check(lib().gemm_select_config_mx_wgrad(out_dtype, rows, M, N, groups, 1 if q_second else 0, buf, len(buf)),
           "gemm_select_config_mx_wgrad")
    return buf.value.decode()
