"""Python binding of the fine-grained FP8 GEMM C-ABI library (``include/fg.h``).

Argument marshalling only: every function takes torch CUDA tensors, checks dtypes and
contiguity, and passes raw device pointers, host-side sizes and the current CUDA stream
to the same-named ``fg_*`` C entry point.  All arithmetic runs in the library's CUDA
kernels; there is no fallback.  Importing fails loudly if ``libfg.so`` has not been
built (``moe_fp8_e4m3_gb300.build.build()``)."""
from __future__ import annotations

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfg.so")

FG_OK = 0
FG_ERR_INVALID_ARG = -1
FG_ERR_UNSUPPORTED = -2
FG_ERR_CUDA = -3
FG_ERR_DEVICE_CONTRACT = -4
FG_ERR_DEVICE_TIMEOUT = -5
FG_BF16 = 0
FG_F32 = 1
FG_SCORE_SOFTMAX = 0
FG_SCORE_SIGMOID = 1

_P = ctypes.c_void_p
_I = ctypes.c_int

_SIGNATURES = {
    "fg_fp8_gemm_nt": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P]),
    "fg_fp8_gemm_nn": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P]),
    "fg_fp8_gemm_tn": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P]),
    "fg_fp8_gemm_tt": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P]),
    "fg_m_grouped_fp8_gemm_nt_contiguous": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P]),
    "fg_m_grouped_fp8_gemm_nn_contiguous": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P]),
    "fg_m_grouped_fp8_gemm_nt_contiguous_swiglu": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "fg_fp8_mqa_logits": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P, _P]),
    "fg_m_grouped_fp8_gemm_nt_masked_swiglu": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "fg_m_grouped_fp8_gemm_nt_masked": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _I, _P, _I, _P]),
    "fg_fp8_fp4_gemm_nt": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P]),
    "fg_m_grouped_fp8_fp4_gemm_nt_contiguous": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P]),
    "fg_m_grouped_fp8_fp4_gemm_nt_masked": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _I, _P, _I, _P]),
    "fg_m_grouped_fp8_fp4_gemm_nt_contiguous_swiglu": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "fg_m_grouped_fp8_fp4_gemm_nt_masked_swiglu": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "fg_k_grouped_fp8_gemm_tn_contiguous": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "fg_quantize_1x128_rows": (_I, [_I, _I, _P, _P, _P, _P]),
    "fg_quantize_128x128_blocks": (_I, [_I, _I, _I, _P, _P, _P, _P]),
    "fg_quantize_1x128_cols": (_I, [_I, _I, _P, _P, _P, _P]),
    "fg_quantize_mxfp4": (_I, [_I, _I, _I, _P, _P, _P, _P]),
    "fg_moe_route": (_I, [_I, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P, _P, _P]),
    "fg_moe_mlp_workspace": (ctypes.c_longlong, [_I, _I, _I, _I]),
    "fg_fp8_moe_mlp": (_I, [_I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P]),
    "fg_fp8_fp4_moe_mlp": (_I, [_I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P]),
    "fg_lora_workspace": (ctypes.c_longlong, [_I, _I, _I, _I]),
    "fg_lora_workspace_for": (ctypes.c_longlong, [_I, _I, _I, _I, _I, _I]),
    "fg_fp8_gemm_nt_lora": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P]),
    "fg_get_mk_alignment_for_contiguous_layout": (_I, []),
    "fg_get_tma_aligned_size": (_I, [_I, _I]),
    "fg_set_num_sms": (None, [_I]),
    "fg_get_num_sms": (_I, []),
    "fg_set_pdl": (None, [_I]),
    "fg_get_pdl": (_I, []),
    "fg_get_device_error": (_I, [_P, ctypes.POINTER(_I)]),
    "fg_status_string": (ctypes.c_char_p, [_I]),
    "fg_debug_inject_stall": (None, [_I, ctypes.c_uint32]),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build the CUDA library first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def _align4(x):
    return (x + 3) // 4 * 4


# Bytes that a call's workspace and scale arrays need, by its sizes: worked out once per size, not once
# per step (the ctypes call alone takes 0.6 us).
@functools.lru_cache(1024)
def _moe_mlp_bytes(t, h, i, e, fp4):
    """(workspace, sfa, sf13, sf2)"""
    if fp4:                                 # a word per 128 K of each row
        sf13, sf2 = h // 128 * _align4(2 * i), i // 128 * _align4(h)
    else:
        sf13, sf2 = (h + 511) // 512 * _align4(2 * i // 128), (i + 511) // 512 * _align4(h // 128)
    return lib.fg_moe_mlp_workspace(t, h, i, e), 4 * ((h + 511) // 512) * _align4(t), 4 * e * sf13, 4 * e * sf2


@functools.lru_cache(1024)
def _lora_bytes(m, n, k, l, r, dtype):
    """(workspace, sfa, sfb)"""
    words = (k + 511) // 512
    return lib.fg_lora_workspace_for(m, n, k, l, r, dtype), 4 * words * _align4(m), 4 * words * _align4((n + 127) // 128)


class FgError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib.fg_status_string(status).decode()} (status {status})")


def _check(status: int, where: str) -> None:
    if status != FG_OK:
        raise FgError(status, where)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        import torch
        # the handle of torch.cuda.current_stream(), without making a Stream object (2.8 us a call)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _fp8(t, name):
    import torch
    if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or not t.is_contiguous() or not t.is_cuda:
        raise TypeError(f"{name} must be a contiguous CUDA uint8/float8_e4m3fn tensor")


def _i32(t, name):
    import torch
    if t.dtype != torch.int32 or not t.is_contiguous() or not t.is_cuda:
        raise TypeError(f"{name} must be a contiguous CUDA int32 tensor")


def _out(t, name):
    import torch
    if t.dtype not in (torch.bfloat16, torch.float32) or not t.is_contiguous() or not t.is_cuda:
        raise TypeError(f"{name} must be a contiguous CUDA bfloat16/float32 tensor")
    return FG_F32 if t.dtype == torch.float32 else FG_BF16


def _c(t):
    import torch
    if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda):
        raise TypeError("c must be a contiguous CUDA float32 tensor")


def fp8_gemm_nt(a, sfa, b, sfb, d, c=None, stream=None) -> None:
    """D = C + A @ B.T.  a [M,K], b [N,K] E4M3; sfa [ceil(K/512), align4(M)] and
    sfb [ceil(K/512), align4(ceil(N/128))] packed UE8M0 int32; d [M,N] BF16/FP32;
    c optional FP32 [M,N] (FP32 d only; may be d)."""
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _c(c)
    code = _out(d, "d")
    m, k = a.shape
    n = b.shape[0]
    _check(lib.fg_fp8_gemm_nt(m, n, k, _ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d),
                              code, _stream(stream)), "fp8_gemm_nt")


def _dense_layout(fn, name, a, sfa, b, sfb, d, c, stream, a_t, b_n):
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _c(c)
    code = _out(d, "d")
    k, m = a.shape if a_t else a.shape[::-1]
    n = b.shape[1] if b_n else b.shape[0]
    _check(fn(m, n, k, _ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d), code, _stream(stream)), name)


def fp8_gemm_nn(a, sfa, b, sfb, d, c=None, stream=None) -> None:
    """D = C + A @ B.  a [M,K], b [K,N] E4M3 (N contiguous); scales, c and d as fp8_gemm_nt."""
    _dense_layout(lib.fg_fp8_gemm_nn, "fp8_gemm_nn", a, sfa, b, sfb, d, c, stream, False, True)


def fp8_gemm_tn(a, sfa, b, sfb, d, c=None, stream=None) -> None:
    """D = C + A.T @ B.  a [K,M] (M contiguous, M % 16 == 0), b [K,N]; scales, c and d as fp8_gemm_nt."""
    _dense_layout(lib.fg_fp8_gemm_tn, "fp8_gemm_tn", a, sfa, b, sfb, d, c, stream, True, True)


def fp8_gemm_tt(a, sfa, b, sfb, d, c=None, stream=None) -> None:
    """D = C + A.T @ B.T.  a [K,M] (M contiguous, M % 16 == 0), b [N,K]; scales, c and d as fp8_gemm_nt."""
    _dense_layout(lib.fg_fp8_gemm_tt, "fp8_gemm_tt", a, sfa, b, sfb, d, c, stream, True, False)


def m_grouped_fp8_gemm_nn_contiguous(a, sfa, b, sfb, m_indices, d, stream=None) -> None:
    """D[m] = A[m] @ B[m_indices[m]] for rows with m_indices[m] >= 0.  a [M_total,K];
    b [G,K,N] (N contiguous); sfb [G, ceil(K/512), align4(ceil(N/128))]; m_indices int32 [M_total]."""
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _i32(m_indices, "m_indices")
    code = _out(d, "d")
    m_total, k = a.shape
    g, _, n = b.shape
    _check(lib.fg_m_grouped_fp8_gemm_nn_contiguous(m_total, n, k, g, _ptr(a), _ptr(sfa), _ptr(b),
                                                   _ptr(sfb), _ptr(m_indices), _ptr(d), code,
                                                   _stream(stream)), "m_grouped_fp8_gemm_nn_contiguous")


def m_grouped_fp8_gemm_nt_contiguous_swiglu(a, sfa, b, sfb, m_indices, q, sfq, stream=None) -> None:
    """Gate-up GEMM + SwiGLU + per-1x128 FP8 requantisation.  a [M_total,K]; b [G,2I,K]
    (I gate rows, then I up rows); q [M_total,I] uint8 (E4M3 codes, out);
    sfq [ceil(I/512), align4(M_total)] int32 packed UE8M0 (out)."""
    _fp8(a, "a"); _fp8(b, "b"); _fp8(q, "q"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _i32(sfq, "sfq")
    _i32(m_indices, "m_indices")
    m_total, k = a.shape
    g, n2, _ = b.shape
    _check(lib.fg_m_grouped_fp8_gemm_nt_contiguous_swiglu(m_total, n2 // 2, k, g, _ptr(a), _ptr(sfa), _ptr(b),
                                                          _ptr(sfb), _ptr(m_indices), _ptr(q), _ptr(sfq),
                                                          _stream(stream)), "m_grouped_fp8_gemm_nt_contiguous_swiglu")


def m_grouped_fp8_gemm_nt_masked_swiglu(a, sfa, b, sfb, masked_m, q, sfq, stream=None) -> None:
    """The masked-layout gate-up GEMM + SwiGLU + requantisation.  a [G,M_max,K]; b [G,2I,K];
    q [G,M_max,I] uint8 (out); sfq [G, ceil(I/512), align4(M_max)] int32 (out)."""
    _fp8(a, "a"); _fp8(b, "b"); _fp8(q, "q"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _i32(sfq, "sfq")
    _i32(masked_m, "masked_m")
    g, m_max, k = a.shape
    n2 = b.shape[1]
    _check(lib.fg_m_grouped_fp8_gemm_nt_masked_swiglu(g, m_max, n2 // 2, k, _ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb),
                                                      _ptr(masked_m), _ptr(q), _ptr(sfq), _stream(stream)),
           "m_grouped_fp8_gemm_nt_masked_swiglu")


def fp8_mqa_logits(q, kv, kv_sf, weights, ks, ke, out, clean_logits=True, stream=None) -> None:
    """Lightning-indexer MQA logits.  q [S,H,D] E4M3 (H=64, D=128); kv [T,D] E4M3;
    kv_sf float32 [T]; weights float32 [S,H]; ks, ke int32 [S]; out float32 [S,T]."""
    import torch
    _fp8(q, "q"); _fp8(kv, "kv"); _i32(ks, "ks"); _i32(ke, "ke")
    for t, name in ((kv_sf, "kv_sf"), (weights, "weights"), (out, "out")):
        if t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda:
            raise TypeError(f"{name} must be a contiguous CUDA float32 tensor")
    s_len, heads, dim = q.shape
    t_len = kv.shape[0]
    _check(lib.fg_fp8_mqa_logits(s_len, t_len, heads, dim, _ptr(q), _ptr(kv), _ptr(kv_sf), _ptr(weights), _ptr(ks),
                                 _ptr(ke), 1 if clean_logits else 0, _ptr(out), _stream(stream)), "fp8_mqa_logits")


def m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, m_indices, d, stream=None) -> None:
    """D[m] = A[m] @ B[m_indices[m]].T for rows with m_indices[m] >= 0.  a [M_total,K];
    b [G,N,K]; sfb [G, ceil(K/512), align4(ceil(N/128))]; m_indices int32 [M_total]."""
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _i32(m_indices, "m_indices")
    code = _out(d, "d")
    m_total, k = a.shape
    g, n, _ = b.shape
    _check(lib.fg_m_grouped_fp8_gemm_nt_contiguous(m_total, n, k, g, _ptr(a), _ptr(sfa), _ptr(b),
                                                   _ptr(sfb), _ptr(m_indices), _ptr(d), code,
                                                   _stream(stream)), "m_grouped_fp8_gemm_nt_contiguous")


def m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, masked_m, d, expected_m=0, stream=None) -> None:
    """D[g, m] = A[g, m] @ B[g].T for m < masked_m[g].  a [G,M_max,K];
    sfa [G, ceil(K/512), align4(M_max)]; b [G,N,K]; masked_m int32 [G] on the device."""
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _i32(masked_m, "masked_m")
    code = _out(d, "d")
    g, m_max, k = a.shape
    n = b.shape[1]
    _check(lib.fg_m_grouped_fp8_gemm_nt_masked(g, m_max, n, k, _ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb),
                                               _ptr(masked_m), int(expected_m), _ptr(d), code,
                                               _stream(stream)), "m_grouped_fp8_gemm_nt_masked")


def _fp4(t, name):
    import torch
    ok = t.dtype == torch.uint8 or t.dtype == getattr(torch, "float4_e2m1fn_x2", torch.uint8)
    if not ok or not t.is_contiguous() or not t.is_cuda:
        raise TypeError(f"{name} must be a contiguous CUDA uint8/float4_e2m1fn_x2 tensor of packed E2M1 pairs")


def fp8_fp4_gemm_nt(a, sfa, b, sfb, d, c=None, stream=None) -> None:
    """D = C + A @ B.T with FP4 B.  a [M,K] E4M3, sfa as fp8_gemm_nt; b [N,K/2] packed E2M1
    (element 2i in the low nibble); sfb [K/128, align4(N)] int32, one UE8M0 scale per 32 K
    elements of each row of B; d [M,N] BF16/FP32; c optional FP32 [M,N] (FP32 d only)."""
    _fp8(a, "a"); _fp4(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _c(c)
    code = _out(d, "d")
    m, k = a.shape
    n = b.shape[0]
    _check(lib.fg_fp8_fp4_gemm_nt(m, n, k, _ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d),
                                  code, _stream(stream)), "fp8_fp4_gemm_nt")


def m_grouped_fp8_fp4_gemm_nt_contiguous(a, sfa, b, sfb, m_indices, d, stream=None) -> None:
    """The M-grouped contiguous GEMM with FP4 B.  a [M_total,K]; b [G,N,K/2] packed E2M1;
    sfb [G, K/128, align4(N)] int32 (1x32 blocks); m_indices int32 [M_total]."""
    _fp8(a, "a"); _fp4(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _i32(m_indices, "m_indices")
    code = _out(d, "d")
    m_total, k = a.shape
    g, n, _ = b.shape
    _check(lib.fg_m_grouped_fp8_fp4_gemm_nt_contiguous(m_total, n, k, g, _ptr(a), _ptr(sfa), _ptr(b),
                                                       _ptr(sfb), _ptr(m_indices), _ptr(d), code,
                                                       _stream(stream)), "m_grouped_fp8_fp4_gemm_nt_contiguous")


def m_grouped_fp8_fp4_gemm_nt_masked(a, sfa, b, sfb, masked_m, d, expected_m=0, stream=None) -> None:
    """The M-grouped masked GEMM with FP4 B.  a [G,M_max,K]; b [G,N,K/2] packed E2M1;
    sfb [G, K/128, align4(N)] int32 (1x32 blocks); masked_m int32 [G] on the device."""
    _fp8(a, "a"); _fp4(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _i32(masked_m, "masked_m")
    code = _out(d, "d")
    g, m_max, k = a.shape
    n = b.shape[1]
    _check(lib.fg_m_grouped_fp8_fp4_gemm_nt_masked(g, m_max, n, k, _ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb),
                                                   _ptr(masked_m), int(expected_m), _ptr(d), code,
                                                   _stream(stream)), "m_grouped_fp8_fp4_gemm_nt_masked")


def m_grouped_fp8_fp4_gemm_nt_contiguous_swiglu(a, sfa, b, sfb, m_indices, q, sfq, stream=None) -> None:
    """The fused gate-up GEMM with FP4 weights.  a [M_total,K]; b [G,2I,K/2] packed E2M1 (I gate
    rows, then I up rows); sfb [G, K/128, align4(2I)] int32 (1x32 blocks); q [M_total,I] uint8
    (out); sfq [ceil(I/512), align4(M_total)] int32 (out)."""
    _fp8(a, "a"); _fp4(b, "b"); _fp8(q, "q"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _i32(sfq, "sfq")
    _i32(m_indices, "m_indices")
    m_total, k = a.shape
    g, n2, _ = b.shape
    _check(lib.fg_m_grouped_fp8_fp4_gemm_nt_contiguous_swiglu(m_total, n2 // 2, k, g, _ptr(a), _ptr(sfa), _ptr(b),
                                                              _ptr(sfb), _ptr(m_indices), _ptr(q), _ptr(sfq),
                                                              _stream(stream)),
           "m_grouped_fp8_fp4_gemm_nt_contiguous_swiglu")


def m_grouped_fp8_fp4_gemm_nt_masked_swiglu(a, sfa, b, sfb, masked_m, q, sfq, stream=None) -> None:
    """The masked fused gate-up GEMM with FP4 weights.  a [G,M_max,K]; b [G,2I,K/2] packed E2M1;
    sfb [G, K/128, align4(2I)]; q [G,M_max,I] uint8 (out); sfq [G, ceil(I/512), align4(M_max)]."""
    _fp8(a, "a"); _fp4(b, "b"); _fp8(q, "q"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _i32(sfq, "sfq")
    _i32(masked_m, "masked_m")
    g, m_max, k = a.shape
    n2 = b.shape[1]
    _check(lib.fg_m_grouped_fp8_fp4_gemm_nt_masked_swiglu(g, m_max, n2 // 2, k, _ptr(a), _ptr(sfa), _ptr(b),
                                                          _ptr(sfb), _ptr(masked_m), _ptr(q), _ptr(sfq),
                                                          _stream(stream)),
           "m_grouped_fp8_fp4_gemm_nt_masked_swiglu")


def k_grouped_fp8_gemm_tn_contiguous(a, sfa, b, sfb, ks, d, c=None, stream=None) -> None:
    """D[g] = C[g] + A_g.T @ B_g.  a [K_total,M], b [K_total,N] E4M3 (MN-major);
    sfa [ceil(K_total/512), align4(M)], sfb [ceil(K_total/512), align4(N)];
    ks int32 [G] on the device; d (and c) FP32 [G,M,N]."""
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _i32(ks, "ks"); _c(c)
    if _out(d, "d") != FG_F32:
        raise TypeError("d must be float32")
    k_total, m = a.shape
    n = b.shape[1]
    g = ks.shape[0]
    _check(lib.fg_k_grouped_fp8_gemm_tn_contiguous(g, m, n, k_total, _ptr(a), _ptr(sfa), _ptr(b),
                                                   _ptr(sfb), _ptr(ks), _ptr(c), _ptr(d),
                                                   _stream(stream)), "k_grouped_fp8_gemm_tn_contiguous")


def _f32(t, name):
    import torch
    if t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda:
        raise TypeError(f"{name} must be a contiguous CUDA float32 tensor")


def quantize_1x128_rows(x, q, sf, stream=None) -> None:
    """x [rows,K] FP32 -> q [rows,K] E4M3 bytes, sf [ceil(K/512), align4(rows)] packed UE8M0."""
    _f32(x, "x"); _fp8(q, "q"); _i32(sf, "sf")
    rows, k = x.shape
    _check(lib.fg_quantize_1x128_rows(rows, k, _ptr(x), _ptr(q), _ptr(sf), _stream(stream)),
           "quantize_1x128_rows")


def quantize_128x128_blocks(w, q, sf, stream=None) -> None:
    """w [G,N,K] (or [N,K]) FP32 -> q E4M3, sf [G, ceil(K/512), align4(ceil(N/128))]."""
    _f32(w, "w"); _fp8(q, "q"); _i32(sf, "sf")
    g, n, k = (1, *w.shape) if w.dim() == 2 else w.shape
    _check(lib.fg_quantize_128x128_blocks(g, n, k, _ptr(w), _ptr(q), _ptr(sf), _stream(stream)),
           "quantize_128x128_blocks")


def quantize_mxfp4(w, q, sf, stream=None) -> None:
    """w [G,N,K] (or [N,K]) FP32 -> q [.., N, K/2] packed E2M1, sf [G, K/128, align4(N)]
    (one UE8M0 scale per 32 K elements of a row): the FP4 weights of the FP8 x FP4 GEMMs."""
    _f32(w, "w"); _fp4(q, "q"); _i32(sf, "sf")
    g, n, k = (1, *w.shape) if w.dim() == 2 else w.shape
    _check(lib.fg_quantize_mxfp4(g, n, k, _ptr(w), _ptr(q), _ptr(sf), _stream(stream)), "quantize_mxfp4")


def quantize_1x128_cols(x, q, sf, stream=None) -> None:
    """x [K,MN] FP32 -> q [K,MN] E4M3, sf [ceil(K/512), align4(MN)] (groups along K)."""
    _f32(x, "x"); _fp8(q, "q"); _i32(sf, "sf")
    k, mn = x.shape
    _check(lib.fg_quantize_1x128_cols(k, mn, _ptr(x), _ptr(q), _ptr(sf), _stream(stream)),
           "quantize_1x128_cols")


_SCORES = {"softmax": FG_SCORE_SOFTMAX, "sigmoid": FG_SCORE_SIGMOID}
_DTYPES = {}


def _dtypes():
    """Dtypes by the letter that _check_all takes, looked up once."""
    import torch
    _DTYPES.update(q={torch.uint8, torch.float8_e4m3fn}, i={torch.int32}, f={torch.float32}, b={torch.bfloat16},
                   p={torch.uint8, getattr(torch, "float4_e2m1fn_x2", torch.uint8)}, o={torch.bfloat16, torch.float32})
    return _DTYPES


_NAMES = {"q": "uint8/float8_e4m3fn", "i": "int32", "f": "float32", "b": "bfloat16", "p": "uint8/float4_e2m1fn_x2 (packed E2M1)",
          "o": "bfloat16/float32"}


def _check_all(*args):
    """(tensor, name, letter) triples in a row: contiguous CUDA tensors of the letter's dtype.  A
    decode step's calls are short on the GPU, so those with many tensors look at them in one
    expression first and come here to name the one that is wrong."""
    kinds = _DTYPES or _dtypes()
    for k in range(0, len(args), 3):
        t = args[k]
        if t.dtype not in kinds[args[k + 2]] or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{args[k + 1]} must be a contiguous CUDA {_NAMES[args[k + 2]]} tensor")


def moe_route(logits, topk_ids, topk_weights, bias=None, score="softmax", n_group=1, topk_group=1,
              renormalize=True, scale=1.0, stream=None) -> None:
    """MoE router.  logits float32 [T,E]; topk_ids int32 [T,topk] and topk_weights float32
    [T,topk] (out); bias float32 [E] added to the scores for the choice only; score "softmax" or
    "sigmoid"; the choice is limited to the topk_group best of n_group groups of experts."""
    _check_all(logits, "logits", "f", topk_ids, "topk_ids", "i", topk_weights, "topk_weights", "f")
    t, e = logits.shape
    shape = topk_ids.shape
    if bias is not None:
        _check_all(bias, "bias", "f")
        if bias.numel() != e:
            raise ValueError("bias must be [E]")
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    if len(shape) != 2 or shape[0] != t or topk_weights.shape != shape:
        raise ValueError("topk_ids and topk_weights must be [T, topk]")
    _check(lib.fg_moe_route(t, e, shape[1], n_group, topk_group, _SCORES[score], 1 if renormalize else 0, scale,
                            logits.data_ptr(), _ptr(bias), topk_ids.data_ptr(), topk_weights.data_ptr(), _stream(stream)),
           "moe_route")


def _workspace(nbytes, device, where):
    import torch
    if nbytes < 0:
        _check(FG_ERR_INVALID_ARG, where)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def moe_mlp_workspace(t, h, i, e, device="cuda"):
    """Zeroed workspace of fp8_moe_mlp / fp8_fp4_moe_mlp for t tokens; reusable, one per concurrent call."""
    return _workspace(lib.fg_moe_mlp_workspace(t, h, i, e), device, "moe_mlp_workspace")


def _moe_mlp(fn, name, letter, a, sfa, w13, sf13, w2, sf2, topk_ids, topk_weights, d, workspace, expert_base, stream):
    kinds = _DTYPES or _dtypes()
    q, w, i32 = kinds["q"], kinds[letter], kinds["i"]
    if not (a.dtype in q and sfa.dtype in i32 and w13.dtype in w and sf13.dtype in i32 and w2.dtype in w and
            sf2.dtype in i32 and topk_ids.dtype in i32 and topk_weights.dtype in kinds["f"] and d.dtype in kinds["o"] and
            a.is_cuda and sfa.is_cuda and w13.is_cuda and sf13.is_cuda and w2.is_cuda and sf2.is_cuda and
            topk_ids.is_cuda and topk_weights.is_cuda and d.is_cuda and
            a.is_contiguous() and sfa.is_contiguous() and w13.is_contiguous() and sf13.is_contiguous() and
            w2.is_contiguous() and sf2.is_contiguous() and topk_ids.is_contiguous() and topk_weights.is_contiguous() and
            d.is_contiguous()):
        _check_all(a, "a", "q", sfa, "sfa", "i", w13, "w13", letter, sf13, "sf13", "i", w2, "w2", letter, sf2, "sf2", "i",
                   topk_ids, "topk_ids", "i", topk_weights, "topk_weights", "f", d, "d", "o")
    shape = a.shape
    t, h = shape
    e, i2, k13 = w13.shape
    i = i2 // 2
    ids = topk_ids.shape
    e2, h2, k2 = w2.shape
    fp4 = letter == "p"                     # two codes a byte
    if (e2 != e or h2 != h or i2 != 2 * i or k13 != (h // 2 if fp4 else h) or k2 != (i // 2 if fp4 else i) or
            len(ids) != 2 or ids[0] != t or topk_weights.shape != ids or d.shape != shape):
        raise ValueError("shapes: a and d [T,H], w13 [E,2I,H], w2 [E,H,I] (FP4: H/2, I/2), topk_ids and topk_weights [T,topk]")
    need, need_a, need13, need2 = _moe_mlp_bytes(t, h, i, e, fp4)
    if sfa.nbytes < need_a or sf13.nbytes < need13 or sf2.nbytes < need2:
        raise ValueError("scales: sfa [ceil(H/512), align4(T)]; sf13 [E, ceil(H/512), align4(2I/128)], sf2 [E, ceil(I/512), "
                         "align4(H/128)] (FP4: [E, H/128, align4(2I)], [E, I/128, align4(H)])")
    if not workspace.is_cuda or not workspace.is_contiguous() or workspace.nbytes < need:
        raise ValueError("workspace must be a contiguous CUDA tensor of at least moe_mlp_workspace(t, h, i, e) bytes")
    st = fn(t, h, i, e, ids[1], expert_base, a.data_ptr(), sfa.data_ptr(), w13.data_ptr(), sf13.data_ptr(), w2.data_ptr(),
            sf2.data_ptr(), topk_ids.data_ptr(), topk_weights.data_ptr(), d.data_ptr(),
            FG_F32 if d.dtype in _DTYPES["f"] else FG_BF16, workspace.data_ptr(), _stream(stream))
    if st != FG_OK:
        _check(st, name)


def fp8_moe_mlp(a, sfa, w13, sf13, w2, sf2, topk_ids, topk_weights, d, workspace, expert_base=0, stream=None) -> None:
    """The whole MoE MLP for at most 128 tokens.  a [T,H] E4M3 with sfa; w13 [E,2I,H] (I gate rows,
    then I up rows) with sf13 [E, ceil(H/512), align4(2I/128)]; w2 [E,H,I] with sf2; topk_ids int32
    and topk_weights float32 [T,topk]; d [T,H] BF16/FP32 (out).  Ids outside [expert_base,
    expert_base + E) are skipped.  workspace from moe_mlp_workspace."""
    _moe_mlp(lib.fg_fp8_moe_mlp, "fp8_moe_mlp", "q", a, sfa, w13, sf13, w2, sf2, topk_ids, topk_weights, d, workspace,
             expert_base, stream)


def fp8_fp4_moe_mlp(a, sfa, w13, sf13, w2, sf2, topk_ids, topk_weights, d, workspace, expert_base=0,
                    stream=None) -> None:
    """fp8_moe_mlp with FP4 weights: w13 [E,2I,H/2] packed E2M1 with sf13 [E, H/128, align4(2I)],
    w2 [E,H,I/2] with sf2 [E, I/128, align4(H)] (one UE8M0 scale per 32 K elements of a row)."""
    _moe_mlp(lib.fg_fp8_fp4_moe_mlp, "fp8_fp4_moe_mlp", "p", a, sfa, w13, sf13, w2, sf2, topk_ids, topk_weights, d,
             workspace, expert_base, stream)


def lora_workspace(m, n, k, r, device="cuda", adapters=None, dtype=None):
    """Zeroed workspace of fp8_gemm_nt_lora; reusable, one per concurrent call.  With the number of
    adapters and D's dtype it holds no more than calls with at most so many and that dtype need."""
    import torch
    if adapters is None and dtype is None:
        nbytes = lib.fg_lora_workspace(m, n, k, r)
    else:
        nbytes = lib.fg_lora_workspace_for(m, n, k, 1024 if adapters is None else adapters, r,
                                           FG_BF16 if dtype == torch.bfloat16 else FG_F32)
    return _workspace(nbytes, device, "lora_workspace")


def fp8_gemm_nt_lora(a, sfa, b, sfb, x, lora_a, lora_b, scaling, ids, d, workspace, stream=None) -> None:
    """D[m] = A[m] @ B.T + scaling[l] * (x[m] @ lora_a[l].T) @ lora_b[l].T with l = ids[m] (-1: no
    adapter).  a, sfa, b, sfb as fp8_gemm_nt; x [M,K], lora_a [L,R,K], lora_b [L,N,R] BF16; scaling
    float32 [L]; ids int32 [M]; d [M,N] BF16/FP32 (out).  workspace from lora_workspace."""
    kinds = _DTYPES or _dtypes()
    q, i32, bf = kinds["q"], kinds["i"], kinds["b"]
    if not (a.dtype in q and sfa.dtype in i32 and b.dtype in q and sfb.dtype in i32 and x.dtype in bf and
            lora_a.dtype in bf and lora_b.dtype in bf and scaling.dtype in kinds["f"] and ids.dtype in i32 and
            d.dtype in kinds["o"] and
            a.is_cuda and sfa.is_cuda and b.is_cuda and sfb.is_cuda and x.is_cuda and lora_a.is_cuda and
            lora_b.is_cuda and scaling.is_cuda and ids.is_cuda and d.is_cuda and
            a.is_contiguous() and sfa.is_contiguous() and b.is_contiguous() and sfb.is_contiguous() and
            x.is_contiguous() and lora_a.is_contiguous() and lora_b.is_contiguous() and scaling.is_contiguous() and
            ids.is_contiguous() and d.is_contiguous()):
        _check_all(a, "a", "q", sfa, "sfa", "i", b, "b", "q", sfb, "sfb", "i", x, "x", "b", lora_a, "lora_a", "b",
                   lora_b, "lora_b", "b", scaling, "scaling", "f", ids, "ids", "i", d, "d", "o")
    shape = a.shape
    m, k = shape
    n, kb = b.shape
    l, r, ka = lora_a.shape
    lb, nb, rb = lora_b.shape
    if (kb != k or x.shape != shape or ka != k or lb != l or nb != n or rb != r or scaling.numel() != l or
            ids.numel() != m or d.shape != (m, n)):
        raise ValueError("shapes: a and x [M,K], b [N,K], lora_a [L,R,K], lora_b [L,N,R], scaling [L], ids [M], d [M,N]")
    code = FG_F32 if d.dtype in _DTYPES["f"] else FG_BF16
    need, need_a, need_b = _lora_bytes(m, n, k, l, r, code)
    if sfa.nbytes < need_a or sfb.nbytes < need_b:
        raise ValueError("scales: sfa [ceil(K/512), align4(M)], sfb [ceil(K/512), align4(ceil(N/128))]")
    if not workspace.is_cuda or not workspace.is_contiguous() or workspace.nbytes < need:
        raise ValueError("workspace must be a contiguous CUDA tensor of at least lora_workspace(m, n, k, r, adapters=L, "
                         "dtype=d.dtype) bytes")
    st = lib.fg_fp8_gemm_nt_lora(m, n, k, l, r, a.data_ptr(), sfa.data_ptr(), b.data_ptr(), sfb.data_ptr(), x.data_ptr(),
                                 lora_a.data_ptr(), lora_b.data_ptr(), scaling.data_ptr(), ids.data_ptr(), d.data_ptr(),
                                 code, workspace.data_ptr(), _stream(stream))
    if st != FG_OK:
        _check(st, "fp8_gemm_nt_lora")


def get_mk_alignment_for_contiguous_layout() -> int:
    return lib.fg_get_mk_alignment_for_contiguous_layout()


def get_tma_aligned_size(x: int, elem_bytes: int) -> int:
    return lib.fg_get_tma_aligned_size(x, elem_bytes)


def set_num_sms(n: int) -> None:
    lib.fg_set_num_sms(n)


def get_num_sms() -> int:
    return lib.fg_get_num_sms()


def set_pdl(enable: bool) -> None:
    """Programmatic dependent launch of the GEMM kernels on (default) or off."""
    lib.fg_set_pdl(1 if enable else 0)


def get_pdl() -> bool:
    return bool(lib.fg_get_pdl())


def get_device_error(stream=None) -> tuple[int, int]:
    """Synchronises the stream; returns (status, raw code) and clears the status word."""
    detail = ctypes.c_int(0)
    st = lib.fg_get_device_error(_stream(stream), ctypes.byref(detail))
    return st, detail.value


def debug_inject_stall(enable: bool, timeout_us: int = 0) -> None:
    lib.fg_debug_inject_stall(1 if enable else 0, timeout_us)
