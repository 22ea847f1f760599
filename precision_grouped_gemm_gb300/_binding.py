"""ctypes binding of libpgg.so: argument marshalling only."""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

PAD = 128
FMT_E4M3, FMT_E2M1 = 1, 2
MODE_FWD, MODE_DGRAD, MODE_WGRAD = 0, 1, 2
EPI_NONE, EPI_SWIGLU = 0, 1
_FMT = {"e4m3": FMT_E4M3, "e2m1": FMT_E2M1, FMT_E4M3: FMT_E4M3, FMT_E2M1: FMT_E2M1}

_P, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float

# name -> argument types (all return int status)
SIGNATURES = {
    "pgg_version": [],
    "pgg_init": [_I32],
    "pgg_read_error": [_P, _P, _P],
    "pgg_grouped_gemm_fwd": [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P],
    "pgg_grouped_gemm_dgrad": [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P],
    "pgg_grouped_gemm_wgrad": [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P],
    "pgg_grouped_gemm_wgrad_accumulate": [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P],
    "pgg_grouped_fc1_swiglu": [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P],
    "pgg_grouped_fc2_dgrad_swiglu_bwd": [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P],
    "pgg_grouped_fc1_swiglu_clamped": [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _F32, _P, _P],
    "pgg_grouped_fc2_dgrad_swiglu_bwd_clamped": [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _F32, _P, _P],
    "pgg_mx_grouped_gemm_clamped": [_I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32,
                                    _F32, _P, _P],
    "pgg_mx_quantize_rowwise": [_P, _I64, _I64, _I32, _P, _P, _P],
    "pgg_mx_quantize_rowwise_blocked": [_P, _I64, _I64, _I32, _P, _P, _P],
    "pgg_mx_quantize_colwise": [_P, _I64, _I64, _P, _I32, _I32, _P, _P, _I64, _P, _P],
    "pgg_mx_grouped_gemm": [_I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64,
                            _I64, _I32, _I64, _P, _P],
    "pgg_moe_permute": [_P, _P, _I64, _I32, _I64, _I32, _P, _P, _P, _P, ctypes.c_size_t, _P, _P],
    "pgg_moe_permute_noalloc": [_P, _P, _I64, _I32, _I64, _I32, _P, _P, _P, _P, _P],
    "pgg_moe_combine": [_P, _P, _P, _P, _I64, _I32, _I64, _P],
    "pgg_fp8_tensor_scale": [_P, _I64, _P, _P],
    "pgg_fp8_quantize_rowwise": [_P, _I64, _I64, _P, _P, _P],
    "pgg_fp8_quantize_colwise": [_P, _I64, _I64, _P, _I32, _P, _P, _I64, _P, _P],
    "pgg_fp8_grouped_gemm": [_I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I64, _F32, _P,
                             ctypes.c_size_t, _P, _P],
    "pgg_moe_combine_bwd": [_P, _P, _P, _P, _P, _P, _I64, _I32, _I64, _P],
    "pgg_add_rmsnorm": [_P, _P, _P, _I64, _I64, _F32, _I32, _P, _P, _P, _P, _P, _P],
    "pgg_add_rmsnorm_bwd_workspace_size": [_I64, _I64, _P],
    "pgg_add_rmsnorm_bwd": [_P, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, ctypes.c_size_t, _P],
    "pgg_moe_route": [_P, _I32, _P, _I64, _I32, _I32, _I32, _I32, _F32, _P, _P, _P],
    "pgg_moe_route_bwd": [_P, _I32, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _F32, _P, _P],
    "pgg_moe_decode_workspace_size": [_I32, _I64, _I32, _I64, _I64, _I32, _P],
    "pgg_moe_decode": [_P, _P, _P, _P, _P, _P, _I64, _I32, _I64, _I64, _I32, _F32, _P, ctypes.c_size_t, _P, _P],
    "pgg_mx_moe_decode": [_I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I64, _I64, _I32, _F32, _P,
                          ctypes.c_size_t, _P, _P],
    "pgg_test_stalled_moe_decode": [_I32, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I64, _I64, _I32, _I64,
                                    ctypes.c_uint64, _P, ctypes.c_size_t, _P, _P],
    "pgg_test_stalled_fwd": [_I32, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I64, ctypes.c_uint64, _P, _P],
}


class PggError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib().pgg_status_string(status).decode() if _LIB is not None else str(status)
        super().__init__(f"{where}: pgg status {status} ({msg})")
        self.status = status


def library_path() -> str:
    return os.path.join(_HERE, "libpgg.so")


def lib():
    """Load libpgg.so (raises if it has not been built: there is no fallback)."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with precision_grouped_gemm_gb300.build.build()")
        L = ctypes.CDLL(path)
        for name, args in SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.pgg_status_string.argtypes = [ctypes.c_int]
        L.pgg_status_string.restype = ctypes.c_char_p
        L.pgg_moe_permute_workspace_size.argtypes = [_I64, _I32]
        L.pgg_moe_permute_workspace_size.restype = ctypes.c_size_t
        L.pgg_fp8_workspace_size.argtypes = [_I64, _I64, _I32, _I64]
        L.pgg_fp8_workspace_size.restype = ctypes.c_size_t
        _LIB = L
    return _LIB


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current stream's handle without building a Stream object (0.2 us instead of 3 us a call on a
# Grace host); torch builds without these two functions take the long way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _raw_device is not None:
            return _raw_stream(_raw_device())
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(st: int, where: str):
    if st != 0:
        raise PggError(st, where)


def _dev(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must live on the CUDA device")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")


def _lens(group_lens):
    if group_lens.dtype != torch.int32:
        raise ValueError("group_lens must be int32")
    return group_lens


def version() -> int:
    return lib().pgg_version()


def init(device: int = 0):
    _check(lib().pgg_init(device), "pgg_init")


def read_error(err, stream=None) -> int:
    out = ctypes.c_int32(0)
    _check(lib().pgg_read_error(_ptr(err), ctypes.byref(out), _stream(stream)), "pgg_read_error")
    return out.value


def grouped_gemm_fwd(X, W, group_lens, Y=None, err=None, stream=None):
    """Y_g = X_g . W_g^T; X [M,K] bf16, W [G,N,K] bf16 -> Y [M,N] bf16."""
    M, K = X.shape
    G, N, _ = W.shape
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _dev(X, W, group_lens, Y, err)
    _check(lib().pgg_grouped_gemm_fwd(_ptr(X), _ptr(W), _ptr(_lens(group_lens)), _ptr(Y), M, N, K, G,
                                      _ptr(err), _stream(stream)), "pgg_grouped_gemm_fwd")
    return Y


def grouped_gemm_dgrad(dY, W, group_lens, dX=None, err=None, stream=None):
    """dX_g = dY_g . W_g; dY [M,N] bf16, W [G,N,K] bf16 -> dX [M,K] bf16."""
    M, N = dY.shape
    G, _, K = W.shape
    if dX is None:
        dX = torch.empty((M, K), dtype=torch.bfloat16, device=dY.device)
    _dev(dY, W, group_lens, dX, err)
    _check(lib().pgg_grouped_gemm_dgrad(_ptr(dY), _ptr(W), _ptr(_lens(group_lens)), _ptr(dX), M, N, K,
                                        G, _ptr(err), _stream(stream)), "pgg_grouped_gemm_dgrad")
    return dX


def grouped_gemm_wgrad(X, dY, group_lens, dW=None, err=None, stream=None):
    """dW_g = dY_g^T . X_g; X [M,K], dY [M,N] bf16 -> dW [G,N,K] bf16 (0 for empty groups)."""
    M, K = X.shape
    N = dY.shape[1]
    G = group_lens.numel()
    if dW is None:
        dW = torch.empty((G, N, K), dtype=torch.bfloat16, device=X.device)
    _dev(X, dY, group_lens, dW, err)
    _check(lib().pgg_grouped_gemm_wgrad(_ptr(X), _ptr(dY), _ptr(_lens(group_lens)), _ptr(dW), M, N, K,
                                        G, _ptr(err), _stream(stream)), "pgg_grouped_gemm_wgrad")
    return dW


def grouped_gemm_wgrad_accumulate(X, dY, group_lens, dW_f32, err=None, stream=None):
    """dW_f32[g] += dY_g^T . X_g in place (fp32 main_grad accumulation); returns dW_f32."""
    M, K = X.shape
    N = dY.shape[1]
    G = group_lens.numel()
    if dW_f32.dtype != torch.float32 or tuple(dW_f32.shape) != (G, N, K):
        raise ValueError("dW_f32 must be float32 [G, N, K]")
    _dev(X, dY, group_lens, dW_f32, err)
    _check(lib().pgg_grouped_gemm_wgrad_accumulate(_ptr(X), _ptr(dY), _ptr(_lens(group_lens)), _ptr(dW_f32), M, N,
                                                   K, G, _ptr(err), _stream(stream)),
           "pgg_grouped_gemm_wgrad_accumulate")
    return dW_f32


def grouped_fc1_swiglu(X, W1, group_lens, A=None, H=None, save_h=True, err=None, stream=None, swiglu_limit=0.0):
    """FC1 + SwiGLU: W1 [G,2I,K] (gate | up) -> A [M,I] and (optionally) H [M,2I];
    swiglu_limit > 0 selects the clamped SwiGLU."""
    M, K = X.shape
    G, I2, _ = W1.shape
    I = I2 // 2
    if A is None:
        A = torch.empty((M, I), dtype=torch.bfloat16, device=X.device)
    if H is None and save_h:
        H = torch.empty((M, 2 * I), dtype=torch.bfloat16, device=X.device)
    _dev(X, W1, group_lens, A, H, err)
    if swiglu_limit:
        _check(lib().pgg_grouped_fc1_swiglu_clamped(_ptr(X), _ptr(W1), _ptr(_lens(group_lens)), _ptr(A), _ptr(H),
                                                    M, I, K, G, swiglu_limit, _ptr(err), _stream(stream)),
               "pgg_grouped_fc1_swiglu_clamped")
    else:
        _check(lib().pgg_grouped_fc1_swiglu(_ptr(X), _ptr(W1), _ptr(_lens(group_lens)), _ptr(A), _ptr(H),
                                            M, I, K, G, _ptr(err), _stream(stream)), "pgg_grouped_fc1_swiglu")
    return A, H


def grouped_fc2_dgrad_swiglu_bwd(dY, W2, H, group_lens, dH=None, err=None, stream=None, swiglu_limit=0.0):
    """dA = dY . W2_g (W2 [G,Hd,I]); dH [M,2I] = SwiGLU backward of dA at the saved H
    (swiglu_limit > 0: of the clamped SwiGLU)."""
    M, Hd = dY.shape
    G, _, I = W2.shape
    if dH is None:
        dH = torch.empty((M, 2 * I), dtype=torch.bfloat16, device=dY.device)
    _dev(dY, W2, H, group_lens, dH, err)
    if swiglu_limit:
        _check(lib().pgg_grouped_fc2_dgrad_swiglu_bwd_clamped(_ptr(dY), _ptr(W2), _ptr(H), _ptr(_lens(group_lens)),
                                                              _ptr(dH), M, Hd, I, G, swiglu_limit, _ptr(err),
                                                              _stream(stream)),
               "pgg_grouped_fc2_dgrad_swiglu_bwd_clamped")
    else:
        _check(lib().pgg_grouped_fc2_dgrad_swiglu_bwd(_ptr(dY), _ptr(W2), _ptr(H), _ptr(_lens(group_lens)),
                                                      _ptr(dH), M, Hd, I, G, _ptr(err), _stream(stream)),
               "pgg_grouped_fc2_dgrad_swiglu_bwd")
    return dH


def mx_quantize_rowwise(x, fmt, codes=None, scales=None, stream=None):
    """bf16 [R,C] -> (codes [R,C] or [R,C/2] u8, scales [R,C/32] u8), blocks along C."""
    R, C = x.shape
    f = _FMT[fmt]
    if codes is None:
        codes = torch.empty((R, C if f == FMT_E4M3 else C // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((R, C // 32), dtype=torch.uint8, device=x.device)
    _dev(x, codes, scales)
    _check(lib().pgg_mx_quantize_rowwise(_ptr(x), R, C, f, _ptr(codes), _ptr(scales), _stream(stream)),
           "pgg_mx_quantize_rowwise")
    return codes, scales


def mx_quantize_rowwise_blocked(x, fmt, codes=None, scales=None, stream=None):
    """bf16 [R,C] (C % 128 == 0) -> (codes as mx_quantize_rowwise, scales [round_up(R,128), C/32]
    bytes in the blocked atom layout): the forward GEMM's weight operand."""
    R, C = x.shape
    f = _FMT[fmt]
    if codes is None:
        codes = torch.empty((R, C if f == FMT_E4M3 else C // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((-(-R // 128) * 128, C // 32), dtype=torch.uint8, device=x.device)
    _dev(x, codes, scales)
    _check(lib().pgg_mx_quantize_rowwise_blocked(_ptr(x), R, C, f, _ptr(codes), _ptr(scales), _stream(stream)),
           "pgg_mx_quantize_rowwise_blocked")
    return codes, scales


def mx_pad_rows(M: int, G: int) -> int:
    """An M_pad that always holds sum(round_up(len_g, PAD)) for any split of M rows in G groups."""
    return -(-(M + G * (PAD - 1)) // PAD) * PAD


def mx_quantize_colwise(x, group_lens, fmt, M_pad=None, codes_t=None, scales_t=None, err=None,
                        stream=None):
    """bf16 [M,C] + group_lens -> transposed codes_t [C,M_pad] (or [C,M_pad/2]) and scales_t
    [round_up(C,128), M_pad/32] bytes in the blocked atom layout (see pgg.h)."""
    M, C = x.shape
    f = _FMT[fmt]
    G = 1 if group_lens is None else group_lens.numel()
    if M_pad is None:
        M_pad = mx_pad_rows(M, G)
    if codes_t is None:
        codes_t = torch.empty((C, M_pad if f == FMT_E4M3 else M_pad // 2), dtype=torch.uint8, device=x.device)
    if scales_t is None:  # blocked atom layout, rows padded to a multiple of 128
        scales_t = torch.empty((-(-C // 128) * 128, M_pad // 32), dtype=torch.uint8, device=x.device)
    _dev(x, group_lens, codes_t, scales_t, err)
    lens = None if group_lens is None else _lens(group_lens)
    _check(lib().pgg_mx_quantize_colwise(_ptr(x), M, C, _ptr(lens), G, f, _ptr(codes_t), _ptr(scales_t),
                                         M_pad, _ptr(err), _stream(stream)), "pgg_mx_quantize_colwise")
    return codes_t, scales_t


def mx_grouped_gemm(mode, fmt, A, SA, B, SB, group_lens, M, N, K, out=None, out2=None, H=None,
                    epilogue=EPI_NONE, M_pad=0, err=None, stream=None, out_q=None, swiglu_limit=0.0):
    """Block-scaled grouped GEMM on MX operands (see pgg.h for the per-mode layouts).

    out_q: optional (codes, scales) receiving the row-wise MX quantization of `out`
    (SwiGLU epilogues only); swiglu_limit > 0 (SwiGLU epilogues) clamps the SwiGLU."""
    f = _FMT[fmt]
    G = group_lens.numel()
    dev = A.device
    if out is None:
        if mode == MODE_FWD:
            shape = (M, N // 2) if epilogue == EPI_SWIGLU else (M, N)
        elif mode == MODE_DGRAD:
            shape = (M, 2 * K) if epilogue == EPI_SWIGLU else (M, K)
        else:
            shape = (G, N, K)
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    qc, qs = out_q if out_q is not None else (None, None)
    _dev(A, SA, B, SB, group_lens, out, out2, H, err, qc, qs)
    if swiglu_limit:
        if epilogue != EPI_SWIGLU:
            raise ValueError("swiglu_limit needs the SwiGLU epilogue")
        _check(lib().pgg_mx_grouped_gemm_clamped(mode, f, _ptr(A), _ptr(SA), _ptr(B), _ptr(SB), _ptr(H),
                                                 _ptr(_lens(group_lens)), _ptr(out), _ptr(out2), _ptr(qc), _ptr(qs),
                                                 M, N, K, G, swiglu_limit, _ptr(err), _stream(stream)),
               "pgg_mx_grouped_gemm_clamped")
    else:
        _check(lib().pgg_mx_grouped_gemm(mode, f, epilogue, _ptr(A), _ptr(SA), _ptr(B), _ptr(SB), _ptr(H),
                                         _ptr(_lens(group_lens)), _ptr(out), _ptr(out2), _ptr(qc), _ptr(qs), M, N,
                                         K, G, M_pad, _ptr(err), _stream(stream)), "pgg_mx_grouped_gemm")
    return out


def fp8_tensor_scale(x, amax_scale=None, stream=None):
    """bf16 tensor (numel % 8 == 0) -> device float32[2] = (s, amax): amax over the finite
    elements, s = 448 / amax (current scaling, see pgg.h)."""
    if amax_scale is None:
        amax_scale = torch.empty(2, dtype=torch.float32, device=x.device)
    _dev(x, amax_scale)
    _check(lib().pgg_fp8_tensor_scale(_ptr(x), x.numel(), _ptr(amax_scale), _stream(stream)),
           "pgg_fp8_tensor_scale")
    return amax_scale


def fp8_quantize_rowwise(x, amax_scale, codes=None, stream=None):
    """bf16 [R, C] -> e4m3 codes [R, C] (u8) with the tensor scale amax_scale[0]."""
    R, C = x.shape
    if codes is None:
        codes = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    _dev(x, amax_scale, codes)
    _check(lib().pgg_fp8_quantize_rowwise(_ptr(x), R, C, _ptr(amax_scale), _ptr(codes), _stream(stream)),
           "pgg_fp8_quantize_rowwise")
    return codes


def fp8_quantize_colwise(x, group_lens, amax_scale, M_pad=None, codes_t=None, err=None, stream=None):
    """bf16 [M, C] + group_lens -> e4m3 codes_t [C, M_pad] in the group-padded column-wise
    layout (the wgrad operand), with the tensor scale amax_scale[0]."""
    M, C = x.shape
    G = 1 if group_lens is None else group_lens.numel()
    if M_pad is None:
        M_pad = mx_pad_rows(M, G)
    if codes_t is None:
        codes_t = torch.empty((C, M_pad), dtype=torch.uint8, device=x.device)
    _dev(x, group_lens, amax_scale, codes_t, err)
    lens = None if group_lens is None else _lens(group_lens)
    _check(lib().pgg_fp8_quantize_colwise(_ptr(x), M, C, _ptr(lens), G, _ptr(amax_scale), _ptr(codes_t), M_pad,
                                          _ptr(err), _stream(stream)), "pgg_fp8_quantize_colwise")
    return codes_t


def fp8_workspace_size(N: int, K: int, G: int, M_pad: int = 0) -> int:
    return lib().pgg_fp8_workspace_size(N, K, G, M_pad)


def fp8_grouped_gemm(mode, A, scale_a, B, scale_b, group_lens, M, N, K, out=None, out2=None, H=None,
                     epilogue=EPI_NONE, M_pad=0, ws=None, err=None, stream=None, swiglu_limit=0.0):
    """FP8 tensor-wise grouped GEMM: the MX operand layouts and epilogues in e4m3, one scale per
    operand (scale_a / scale_b are the operands' amax_scale tensors; see pgg.h)."""
    G = group_lens.numel()
    dev = A.device
    if out is None:
        if mode == MODE_FWD:
            shape = (M, N // 2) if epilogue == EPI_SWIGLU else (M, N)
        elif mode == MODE_DGRAD:
            shape = (M, 2 * K) if epilogue == EPI_SWIGLU else (M, K)
        else:
            shape = (G, N, K)
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    _dev(A, scale_a, B, scale_b, group_lens, out, out2, H, ws, err)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().pgg_fp8_grouped_gemm(mode, epilogue, _ptr(A), _ptr(scale_a), _ptr(B), _ptr(scale_b), _ptr(H),
                                      _ptr(_lens(group_lens)), _ptr(out), _ptr(out2), M, N, K, G, M_pad,
                                      swiglu_limit, _ptr(ws), ws_bytes, _ptr(err), _stream(stream)),
           "pgg_fp8_grouped_gemm")
    return out


def moe_permute_workspace_size(T: int, E: int) -> int:
    return int(lib().pgg_moe_permute_workspace_size(T, E))


def moe_permute(topk_ids, X, E, Xs=None, group_lens=None, pos=None, ws=None, err=None, stream=None):
    """topk_ids [T,k] int32 (+ X [T,H] bf16 or None) -> (Xs [T*k,H], group_lens [E], pos [T,k])."""
    T, k = topk_ids.shape
    if topk_ids.dtype != torch.int32:
        raise ValueError("topk_ids must be int32")
    dev = topk_ids.device
    H = 0 if X is None else X.shape[1]
    if X is not None and Xs is None:
        Xs = torch.empty((T * k, H), dtype=torch.bfloat16, device=dev)
    if group_lens is None:
        group_lens = torch.empty(E, dtype=torch.int32, device=dev)
    if pos is None:
        pos = torch.empty((T, k), dtype=torch.int32, device=dev)
    nbytes = moe_permute_workspace_size(T, E)
    if ws is None:
        ws = torch.empty(max(1, nbytes // 4), dtype=torch.int32, device=dev)
    _dev(topk_ids, X, Xs, group_lens, pos, ws, err)
    _check(lib().pgg_moe_permute(_ptr(topk_ids), _ptr(X), T, k, H, E, _ptr(Xs), _ptr(group_lens), _ptr(pos),
                                 _ptr(ws), ws.numel() * ws.element_size(), _ptr(err), _stream(stream)),
           "pgg_moe_permute")
    return Xs, group_lens, pos


def moe_combine(Ys, pos, w=None, out=None, stream=None):
    """out[t] = sum_j w[t,j] * Ys[pos[t,j]] (w None: weight 1, the permute backward)."""
    T, k = pos.shape
    H = Ys.shape[1]
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=Ys.device)
    if w is not None and w.dtype != torch.float32:
        raise ValueError("w must be float32")
    _dev(Ys, pos, w, out)
    _check(lib().pgg_moe_combine(_ptr(Ys), _ptr(pos), _ptr(w), _ptr(out), T, k, H, _stream(stream)),
           "pgg_moe_combine")
    return out


def moe_combine_bwd(dOut, Ys, pos, w, dYs=None, dw=None, stream=None):
    """-> (dYs [R,H] bf16 with dYs[pos[t,j]] = w[t,j] dOut[t], dw [T,k] fp32)."""
    T, k = pos.shape
    H = dOut.shape[1]
    if dYs is None:
        dYs = torch.empty_like(Ys)
    if dw is None:
        dw = torch.empty((T, k), dtype=torch.float32, device=dOut.device)
    if w.dtype != torch.float32:
        raise ValueError("w must be float32")
    _dev(dOut, Ys, pos, w, dYs, dw)
    _check(lib().pgg_moe_combine_bwd(_ptr(dOut), _ptr(Ys), _ptr(pos), _ptr(w), _ptr(dYs), _ptr(dw), T, k, H,
                                     _stream(stream)), "pgg_moe_combine_bwd")
    return dYs, dw


def _in(t, what, dtype, shape):
    """The address of a caller's tensor of this type and shape (None for None); _dev checks the rest
    of what the caller has given."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise ValueError(f"{what} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}")
    return t.data_ptr()


def _new(make, shape, dtype, device, stream):
    """A new tensor in the order of the call's stream (None: the current one)."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _out(t, what, dtype, shape, device, stream):
    """The caller's output tensor or a new one, and its address."""
    if t is None:
        t = (torch.empty(shape, dtype=dtype, device=device) if stream is None
             else _new(torch.empty, shape, dtype, device, stream))
        return t, t.data_ptr()
    return t, _in(t, what, dtype, shape)


def _size_of(name, *args):
    out = ctypes.c_size_t(0)
    _check(getattr(lib(), name)(*args, ctypes.byref(out)), name)
    return out.value


_BF, _F, _I, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _scratch(ws):
    """Address and bytes of a workspace."""
    return ws.data_ptr(), ws.numel() * ws.element_size()


def add_rmsnorm(x, residual, gamma, eps=1e-6, fmt=None, h=None, y=None, codes=None, scales=None, rstd=None,
                save_y=True, save_rstd=True, stream=None):
    """s = x + residual (residual may be None), y = s / sqrt(mean(s^2) + eps) * gamma; x [R,C] bf16.

    -> (h = bf16(s), y, codes, scales, rstd): y None with save_y=False, codes / scales (the
    row-wise MX operand in `fmt`) None without fmt, rstd None with save_rstd=False."""
    given = x, residual, gamma, h, y, codes, scales, rstd
    R, C = shape = x.shape
    dev = x.device
    f = 0 if fmt is None else _FMT[fmt]
    px, pr = _in(x, "x", _BF, shape), _in(residual, "residual", _BF, shape)
    pg = _in(gamma, "gamma", _BF, (C,))
    h, ph = _out(h, "h", _BF, shape, dev, stream)
    py = pc = ps = pd = None
    if save_y or y is not None:
        y, py = _out(y, "y", _BF, shape, dev, stream)
    if f:
        codes, pc = _out(codes, "codes", _U8, (R, C if f == FMT_E4M3 else C // 2), dev, stream)
        scales, ps = _out(scales, "scales", _U8, (R, C // 32), dev, stream)
    elif codes is not None or scales is not None:
        raise ValueError("codes and scales need fmt")
    if save_rstd or rstd is not None:
        rstd, pd = _out(rstd, "rstd", _F, (R,), dev, stream)
    _dev(*given)
    _check(lib().pgg_add_rmsnorm(px, pr, pg, R, C, eps, f, ph, py, pc, ps, pd, _stream(stream)), "pgg_add_rmsnorm")
    return h, y, codes, scales, rstd


@functools.lru_cache(maxsize=1024)
def add_rmsnorm_bwd_workspace_size(R: int, C: int) -> int:
    return _size_of("pgg_add_rmsnorm_bwd_workspace_size", R, C)


def add_rmsnorm_bwd(dy, dh, h, gamma, rstd, dx=None, dgamma=None, ws=None, stream=None):
    """Backward of add_rmsnorm: dy [R,C] bf16, dh the gradient of h (or None), h and rstd as saved
    -> (dx [R,C] bf16, the gradient of x and of residual, dgamma [C] fp32)."""
    given = dy, dh, h, gamma, rstd, dx, dgamma, ws
    R, C = shape = dy.shape
    dev = dy.device
    py, pd, ph = _in(dy, "dy", _BF, shape), _in(dh, "dh", _BF, shape), _in(h, "h", _BF, shape)
    pg, pr = _in(gamma, "gamma", _BF, (C,)), _in(rstd, "rstd", _F, (R,))
    dx, px = _out(dx, "dx", _BF, shape, dev, stream)
    dgamma, pw = _out(dgamma, "dgamma", _F, (C,), dev, stream)
    if ws is None:
        ws = _new(torch.empty, max(16, add_rmsnorm_bwd_workspace_size(R, C)), _U8, dev, stream)
    _dev(*given)
    _check(lib().pgg_add_rmsnorm_bwd(py, pd, ph, pg, pr, R, C, px, pw, *_scratch(ws), _stream(stream)),
           "pgg_add_rmsnorm_bwd")
    return dx, dgamma


_DTYPE = {torch.float32: 0, torch.bfloat16: 1}
_SCORE = {"softmax": 0, "sigmoid": 1}


def _route_kind(logits, score):
    if logits.dtype not in _DTYPE:
        raise ValueError("logits must be float32 or bfloat16")
    if score not in _SCORE:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    return _DTYPE[logits.dtype], _SCORE[score]


def moe_route(logits, k, bias=None, score="softmax", renormalize=True, scale=1.0, ids=None, w=None, stream=None):
    """Top-k routing of gate logits [T,E] (fp32 or bf16) -> (topk_ids [T,k] int32, w [T,k] fp32).

    bias [E] fp32 is added for the choice only (-inf masks an expert); see pgg.h."""
    given = logits, bias, ids, w
    T, E = shape = logits.shape
    dtype, kind = _route_kind(logits, score)
    pl, pb = _in(logits, "logits", logits.dtype, shape), _in(bias, "bias", _F, (E,))
    ids, pi = _out(ids, "ids", _I, (T, k), logits.device, stream)
    w, pw = _out(w, "w", _F, (T, k), logits.device, stream)
    _dev(*given)
    _check(lib().pgg_moe_route(pl, dtype, pb, T, E, k, kind, int(renormalize), scale, pi, pw, _stream(stream)),
           "pgg_moe_route")
    return ids, w


def moe_route_bwd(logits, ids, dw, bias=None, score="softmax", renormalize=True, scale=1.0, dlogits=None,
                  stream=None):
    """dlogits [T,E] (the logits' type) from dw [T,k] at the ids of moe_route."""
    given = logits, bias, ids, dw, dlogits
    T, E = shape = logits.shape
    k = ids.shape[1]
    dtype, kind = _route_kind(logits, score)
    pl, pb = _in(logits, "logits", logits.dtype, shape), _in(bias, "bias", _F, (E,))
    pi, pw = _in(ids, "ids", _I, (T, k)), _in(dw, "dw", _F, (T, k))
    dlogits, pd = _out(dlogits, "dlogits", logits.dtype, shape, logits.device, stream)
    _dev(*given)
    _check(lib().pgg_moe_route_bwd(pl, dtype, pb, pi, pw, T, E, k, kind, int(renormalize), scale, pd,
                                   _stream(stream)), "pgg_moe_route_bwd")
    return dlogits


@functools.lru_cache(maxsize=1024)
def moe_decode_workspace_size(T: int, k: int, H: int, I: int, E: int, fmt=None) -> int:
    return _size_of("pgg_moe_decode_workspace_size", 0 if fmt is None else _FMT[fmt], T, k, H, I, E)


def moe_decode_workspace(T: int, k: int, H: int, I: int, E: int, fmt=None, device="cuda"):
    """A zeroed workspace for moe_decode (fmt None) / mx_moe_decode calls of up to these sizes."""
    return torch.zeros(moe_decode_workspace_size(T, k, H, I, E, fmt), dtype=torch.uint8, device=device)


def moe_decode(X, ids, w, W1, W2, out=None, swiglu_limit=0.0, ws=None, err=None, stream=None):
    """A whole expert layer for T <= 128 tokens: X [T,H] bf16, ids [T,k] int32, w [T,k] fp32 (or None),
    W1 [E,2I,H], W2 [E,H,I] bf16 -> out [T,H] bf16.  ws: a moe_decode_workspace kept between calls
    (None: one is made and zeroed for this call: 42 MB and more, as long as a small layer takes)."""
    given = X, ids, w, W1, W2, out, ws, err
    T, H = shape = X.shape
    E, _, I = W2.shape
    k = ids.shape[1]
    px, pi, pw = _in(X, "X", _BF, shape), _in(ids, "ids", _I, (T, k)), _in(w, "w", _F, (T, k))
    p1, p2 = _in(W1, "W1", _BF, (E, 2 * I, H)), _in(W2, "W2", _BF, (E, H, I))
    out, po = _out(out, "out", _BF, shape, X.device, stream)
    if ws is None:
        ws = _new(torch.zeros, moe_decode_workspace_size(T, k, H, I, E), _U8, X.device, stream)
    pe = None if err is None else _in(err, "err", _I, err.shape)
    _dev(*given)
    _check(lib().pgg_moe_decode(px, pi, pw, p1, p2, po, T, k, H, I, E, swiglu_limit, *_scratch(ws), pe,
                                _stream(stream)), "pgg_moe_decode")
    return out


def mx_moe_decode(fmt, X, SX, ids, w, W1, SW1, W2, SW2, out=None, swiglu_limit=0.0, ws=None, err=None, stream=None):
    """moe_decode on MX operands: X / SX row-wise codes and scales [T, .] (add_rmsnorm or
    mx_quantize_rowwise), W1 [E*2I, .] and W2 [E*H, .] codes with blocked scales
    (mx_quantize_rowwise_blocked).  ws: as there."""
    given = X, SX, ids, w, W1, SW1, W2, SW2, out, ws, err
    f = _FMT[fmt]
    per = 1 if f == FMT_E4M3 else 2  # elements of a byte
    T, H = X.shape[0], X.shape[1] * per
    I = W2.shape[1] * per
    E = W2.shape[0] // H
    k = ids.shape[1]
    px, ps = _in(X, "X", _U8, X.shape), _in(SX, "SX", _U8, (T, H // 32))
    pi, pw = _in(ids, "ids", _I, (T, k)), _in(w, "w", _F, (T, k))
    p1, p2 = _in(W1, "W1", _U8, (E * 2 * I, H // per)), _in(W2, "W2", _U8, (E * H, I // per))
    q1, q2 = _in(SW1, "SW1", _U8, SW1.shape), _in(SW2, "SW2", _U8, SW2.shape)
    if SW1.numel() < E * 2 * I * (H // 32) or SW2.numel() < E * H * (I // 32):
        raise ValueError("SW1 / SW2 are too small for W1 / W2")
    out, po = _out(out, "out", _BF, (T, H), X.device, stream)
    if ws is None:
        ws = _new(torch.zeros, moe_decode_workspace_size(T, k, H, I, E, f), _U8, X.device, stream)
    pe = None if err is None else _in(err, "err", _I, err.shape)
    _dev(*given)
    _check(lib().pgg_mx_moe_decode(f, px, ps, pi, pw, p1, q1, p2, q2, po, T, k, H, I, E, swiglu_limit,
                                   *_scratch(ws), pe, _stream(stream)), "pgg_mx_moe_decode")
    return out
