"""Python binding of libbwta.so (include/bwta.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libbwta.so. PyTorch provides device memory and the current CUDA
stream. There is no CPU fallback: importing works anywhere, but every call
raises if the compiled library is missing or no CUDA device is present.

Bit planes are returned as int32 tensors holding the uint32 words
(bit i of word w is element 32*w + i).
"""
from __future__ import annotations

import ctypes as C
import functools
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbwta.so")
MB_LIB_PATH = os.path.join(_HERE, "libbwta_microbench.so")

BWTA_OK, BWTA_ERR_INVALID_ARG, BWTA_ERR_UNSUPPORTED, BWTA_ERR_ALIGNMENT, BWTA_ERR_CUDA = range(5)
STATUS_NONFINITE, STATUS_TIMEOUT, STATUS_DRAIN = 0x1, 0x2, 0x4
STATUS_BAD_PAGE, STATUS_NO_PAGE = 0x8, 0x10
KV_F16, KV_E4M3 = 0, 1
TERNARY, BINARY = 0, 1
ERROR_NAMES = {1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "ALIGNMENT", 4: "CUDA"}

EXPORTS = ["bwta_pack_weights", "bwta_quantize_pack_acts", "bwta_quantize_pack_acts_ex",
           "bwta_gemm", "bwta_gemm_ex", "bwta_gemm_tc",
           "bwta_linear_decode", "bwta_attn_scores", "billm_pack_weights", "billm_gemm",
           "bwta_linear_decode_batched", "bwta_attn_softmax_ternarize", "bwta_attn_av",
           "bwta_kv_append", "bwta_attn_decode_paged", "bwta_attn_prompt_paged",
           "bwta_kv_reserve", "bwta_kv_free", "bwta_kv_fork", "bwta_kv_compact",
           "bwta_kv_copy_pages",
           "bwta_selftest_gemm_timeout", "bwta_version"]
GEMM_WEIGHTS_READY = 0x1


class BwtaError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} returned {code} ({ERROR_NAMES.get(code, '?')})")
        self.code = code


class BillmWeightsC(C.Structure):
    _fields_ = [("sign", C.c_void_p), ("gmap", C.c_void_p), ("res", C.c_void_p),
                ("sal", C.c_void_p), ("bscale", C.c_void_p), ("N", C.c_int64),
                ("K", C.c_int64), ("ldw_words", C.c_int64), ("block", C.c_int64),
                ("n_sal", C.c_int64)]


class DecodeJobC(C.Structure):
    _fields_ = [("X", C.c_void_p), ("M", C.c_int64), ("K", C.c_int64), ("ldX", C.c_int64),
                ("wbits", C.c_void_p), ("wscale", C.c_void_p), ("N", C.c_int64),
                ("ldw_words", C.c_int64), ("group", C.c_int64), ("Y", C.c_void_p),
                ("ldY", C.c_int64), ("dots", C.c_void_p), ("ldD", C.c_int64)]


class KvCacheC(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("num_pages", C.c_int64), ("page_size", C.c_int64),
                ("n_kv_heads", C.c_int64), ("head_dim", C.c_int64), ("page_stride", C.c_int64),
                ("scale_stride", C.c_int64), ("type", C.c_int32)]


class KvTableC(C.Structure):
    _fields_ = [("pages", C.c_void_p), ("ld", C.c_int64), ("max_pages", C.c_int64),
                ("n_slots", C.c_int64), ("kv_len", C.c_void_p), ("refcount", C.c_void_p)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libbwta.so (raises FileNotFoundError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is missing: run `python -m binarized_transformer_b200.build`")
    lib = C.CDLL(path)
    vp, i64, ci, cf = C.c_void_p, C.c_int64, C.c_int, C.c_float
    lib.bwta_pack_weights.argtypes = [vp, i64, i64, i64, i64, vp, i64, vp, vp, vp]
    lib.bwta_quantize_pack_acts.argtypes = [vp, i64, i64, i64, ci, cf, vp, vp, i64, vp, vp, vp]
    lib.bwta_quantize_pack_acts_ex.argtypes = [vp, i64, i64, i64, ci, cf, vp, vp, i64, vp, i64, vp,
                                               vp, vp]
    lib.bwta_gemm_tc.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, vp, i64, vp, i64,
                                 vp, vp]
    lib.bwta_gemm.argtypes = [vp, vp, vp, i64, i64, vp, vp, i64, i64, i64, i64, vp, i64, vp, i64,
                              vp, vp]
    lib.bwta_gemm_ex.argtypes = [vp, vp, vp, i64, i64, vp, vp, i64, i64, i64, i64, vp, i64, vp,
                                 i64, C.c_uint32, vp, vp]
    lib.bwta_linear_decode.argtypes = [vp, i64, i64, i64, ci, cf, vp, vp, i64, i64, i64, vp, i64,
                                       vp, i64, C.c_uint32, vp, vp]
    lib.bwta_attn_scores.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, vp, vp]
    lib.bwta_attn_softmax_ternarize.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64,
                                                cf, vp, vp, i64, vp, vp]
    lib.bwta_attn_av.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, vp, vp]
    lib.billm_pack_weights.argtypes = [vp, i64, ci, C.POINTER(BillmWeightsC), vp, vp]
    lib.billm_gemm.argtypes = [vp, i64, i64, C.POINTER(BillmWeightsC), vp, i64, vp, vp]
    lib.bwta_linear_decode_batched.argtypes = [C.POINTER(DecodeJobC), i64, ci, cf, C.c_uint32, vp,
                                               vp]
    lib.bwta_selftest_gemm_timeout.argtypes = [vp, vp, vp, i64, i64, vp, vp, i64, i64, i64, i64,
                                               vp, i64, vp, i64, i64, vp, vp]
    kc, kt = C.POINTER(KvCacheC), C.POINTER(KvTableC)
    lib.bwta_kv_append.argtypes = [kc, kt, vp, i64, vp, i64, vp, i64, vp, i64, ci, vp, vp]
    lib.bwta_attn_decode_paged.argtypes = [kc, kt, vp, i64, vp, i64, i64, cf, i64, i64, vp, i64, vp,
                                           i64, vp, vp]
    lib.bwta_attn_prompt_paged.argtypes = [kc, kt, vp, i64, vp, i64, vp, i64, i64, cf, i64, i64, vp,
                                           i64, vp, vp]
    lib.bwta_kv_reserve.argtypes = [kt, i64, i64, vp, vp, i64, vp, vp]
    lib.bwta_kv_free.argtypes = [kt, i64, i64, vp, i64, vp, vp]
    lib.bwta_kv_fork.argtypes = [kc, i64, kt, vp, vp, i64, vp, i64, vp, vp]
    lib.bwta_kv_compact.argtypes = [kc, i64, kt, vp, vp, i64, vp, vp]
    lib.bwta_kv_copy_pages.argtypes = [kc, kc, i64, vp, vp, i64, vp, i64, vp, vp]
    lib.bwta_attn_decode_workspace.argtypes = [i64, i64, i64]
    lib.bwta_attn_decode_workspace.restype = i64
    lib.bwta_kv_pages_workspace.argtypes = [i64, i64]
    lib.bwta_kv_pages_workspace.restype = i64
    lib.bwta_version.restype = C.c_char_p
    for name in EXPORTS[:-1]:
        getattr(lib, name).restype = C.c_int
    _lib = lib
    return lib


def _L():
    if not torch.cuda.is_available():
        raise RuntimeError("libbwta needs a CUDA device; there is no CPU fallback")
    return load_library()


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream():
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(fn, rc):
    if rc != BWTA_OK:
        raise BwtaError(fn, rc)


def _row_stride(t: torch.Tensor) -> int:
    """Leading dimension of a row-major 2-D tensor (a single row may carry any stride)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def ld_words_for(K: int) -> int:
    """Smallest legal row stride in words: ceil(K/32) rounded up to a multiple of 4."""
    return ((K + 31) // 32 + 3) // 4 * 4


def new_status(device=None):
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def version() -> str:
    return load_library().bwta_version().decode()


# ------------------------------------------------------------------ BWTA
def bwta_pack_weights(W: torch.Tensor, group: int = 0, ld_words: int | None = None,
                      status: torch.Tensor | None = None):
    """fp32 W [N, K] (cuda) -> (wbits int32 [N, ld_words], wscale fp32 [N, G])."""
    lib = _L()
    assert W.is_cuda and W.dtype == torch.float32 and W.dim() == 2 and W.stride(1) == 1
    N, K = W.shape
    ld = ld_words or ld_words_for(K)
    G = -(-K // group) if group else 1
    wbits = torch.empty((N, ld), dtype=torch.int32, device=W.device)
    wscale = torch.empty((N, G), dtype=torch.float32, device=W.device)
    _check("bwta_pack_weights", lib.bwta_pack_weights(
        _ptr(W), N, K, _row_stride(W), group, _ptr(wbits), ld, _ptr(wscale), _ptr(status), _stream()))
    return wbits, wscale


def bwta_quantize_pack_acts(X: torch.Tensor, mode: int = TERNARY, thresh_ratio: float = 0.5,
                            ld_words: int | None = None, status: torch.Tensor | None = None,
                            out=None):
    """fp16 X [M, K] (cuda) -> (mask int32 [M, ld], sign int32 [M, ld], scale fp32 [M])."""
    lib = _L()
    assert X.is_cuda and X.dtype == torch.float16 and X.dim() == 2 and X.stride(1) == 1
    M, K = X.shape
    ld = ld_words or ld_words_for(K)
    if out is None:
        mask = torch.empty((M, ld), dtype=torch.int32, device=X.device)
        sign = torch.empty((M, ld), dtype=torch.int32, device=X.device)
        scale = torch.empty((M,), dtype=torch.float32, device=X.device)
    else:
        mask, sign, scale = out
    _check("bwta_quantize_pack_acts", lib.bwta_quantize_pack_acts(
        _ptr(X), M, K, _row_stride(X), mode, thresh_ratio, _ptr(mask), _ptr(sign), ld, _ptr(scale),
        _ptr(status), _stream()))
    return mask, sign, scale


def e4m3_ld_for(K: int) -> int:
    """Row stride in bytes of E4M3 activations for the tensor-core GEMM."""
    return ld_words_for(K) * 32


def bwta_quantize_pack_acts_ex(X: torch.Tensor, mode: int = TERNARY, thresh_ratio: float = 0.5,
                               planes: bool = True, e4m3: bool = True, status=None, out=None):
    """fp16 X [M, K] -> (mask, sign or None, E4M3 uint8 [M, 32*ld] or None, scale [M])."""
    lib = _L()
    assert X.is_cuda and X.dtype == torch.float16 and X.dim() == 2 and X.stride(1) == 1
    M, K = X.shape
    ld = ld_words_for(K)
    if out is None:
        mask = torch.empty((M, ld), dtype=torch.int32, device=X.device) if planes else None
        sign = torch.empty((M, ld), dtype=torch.int32, device=X.device) if planes else None
        a8 = torch.empty((M, 32 * ld), dtype=torch.uint8, device=X.device) if e4m3 else None
        scale = torch.empty((M,), dtype=torch.float32, device=X.device)
    else:
        mask, sign, a8, scale = out
    _check("bwta_quantize_pack_acts_ex", lib.bwta_quantize_pack_acts_ex(
        _ptr(X), M, K, _row_stride(X), mode, thresh_ratio, _ptr(mask), _ptr(sign), ld, _ptr(a8),
        a8.shape[1] if a8 is not None else 0, _ptr(scale), _ptr(status), _stream()))
    return mask, sign, a8, scale


def bwta_gemm_tc(a_e4m3, a_scale, wbits, wscale, K: int, group: int = 0, want_y: bool = True,
                 want_dots: bool = False, status=None, out=None):
    """Tensor-core GEMM on E4M3 activations. Returns (Y fp32 [M, N] or None, dots or None)."""
    lib = _L()
    M, ld8 = a_e4m3.shape
    N, ldw = wbits.shape
    if out is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=a_e4m3.device) if want_y else None
        D = torch.empty((M, N), dtype=torch.int32, device=a_e4m3.device) if want_dots else None
    else:
        Y, D = out
    _check("bwta_gemm_tc", lib.bwta_gemm_tc(
        _ptr(a_e4m3), ld8, _ptr(a_scale), M, _ptr(wbits), _ptr(wscale), N, ldw, K, group, _ptr(Y),
        _row_stride(Y) if Y is not None else N, _ptr(D), _row_stride(D) if D is not None else N,
        _ptr(status), _stream()))
    return Y, D


def bwta_gemm(a_mask, a_sign, a_scale, wbits, wscale, K: int, group: int = 0,
              want_y: bool = True, want_dots: bool = False, status=None, out=None,
              flags: int = 0):
    """Bit-packed GEMM. Returns (Y fp32 [M, N] or None, dots int32 [M, N] or None).
    flags=GEMM_WEIGHTS_READY (weights complete before the call) goes through
    bwta_gemm_ex; 0 through bwta_gemm."""
    lib = _L()
    M, lda = a_mask.shape
    N, ldw = wbits.shape
    if out is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=a_mask.device) if want_y else None
        D = torch.empty((M, N), dtype=torch.int32, device=a_mask.device) if want_dots else None
    else:
        Y, D = out
    ldY = _row_stride(Y) if Y is not None else N
    ldD = _row_stride(D) if D is not None else N
    if flags:
        rc = lib.bwta_gemm_ex(_ptr(a_mask), _ptr(a_sign), _ptr(a_scale), M, lda, _ptr(wbits),
                              _ptr(wscale), N, ldw, K, group, _ptr(Y), ldY, _ptr(D), ldD, flags,
                              _ptr(status), _stream())
        _check("bwta_gemm_ex", rc)
    else:
        _check("bwta_gemm", lib.bwta_gemm(
            _ptr(a_mask), _ptr(a_sign), _ptr(a_scale), M, lda, _ptr(wbits), _ptr(wscale), N, ldw,
            K, group, _ptr(Y), ldY, _ptr(D), ldD, _ptr(status), _stream()))
    return Y, D


def bwta_selftest_gemm_timeout(a_mask, a_sign, a_scale, wbits, wscale, K: int, group: int = 0,
                               wait_limit_ns: int = 1_000_000, status=None, out=None):
    """Failure-path self-test: the tiled GEMM with a wait that is made to run
    out after wait_limit_ns. Returns the status tensor (BWTA_STATUS_TIMEOUT set)."""
    lib = _L()
    M, lda = a_mask.shape
    N, ldw = wbits.shape
    status = new_status(a_mask.device) if status is None else status
    if out is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=a_mask.device)
        D = None
    else:
        Y, D = out
    _check("bwta_selftest_gemm_timeout", lib.bwta_selftest_gemm_timeout(
        _ptr(a_mask), _ptr(a_sign), _ptr(a_scale), M, lda, _ptr(wbits), _ptr(wscale), N, ldw, K,
        group, _ptr(Y), _row_stride(Y) if Y is not None else N, _ptr(D),
        _row_stride(D) if D is not None else N, wait_limit_ns, _ptr(status), _stream()))
    return status


def bwta_linear_decode(X, wbits, wscale, group: int = 0, mode: int = TERNARY,
                       thresh_ratio: float = 0.5, want_y: bool = True, want_dots: bool = False,
                       flags: int = 0, status=None, out=None):
    """Fused decode: fp16 X [M<=8, K] -> ternarize in-kernel -> x packed weights.
    Returns (Y fp32 [M, N] or None, dots int32 [M, N] or None)."""
    lib = _L()
    assert X.is_cuda and X.dtype == torch.float16 and X.dim() == 2 and X.stride(1) == 1
    M, K = X.shape
    N, ldw = wbits.shape
    if out is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=X.device) if want_y else None
        D = torch.empty((M, N), dtype=torch.int32, device=X.device) if want_dots else None
    else:
        Y, D = out
    _check("bwta_linear_decode", lib.bwta_linear_decode(
        _ptr(X), M, K, _row_stride(X), mode, thresh_ratio, _ptr(wbits), _ptr(wscale), N, ldw, group,
        _ptr(Y), _row_stride(Y) if Y is not None else N, _ptr(D),
        _row_stride(D) if D is not None else N, flags, _ptr(status), _stream()))
    return Y, D


def decode_jobs(jobs, want_dots: bool = False):
    """C descriptors for bwta_linear_decode_batched. Each job is a tuple
    (X fp16 [M, K], wbits, wscale, group) or (X, wbits, wscale, group, Y, dots)
    with preallocated outputs (either may be None). Returns (array, outputs)."""
    arr = (DecodeJobC * max(1, len(jobs)))()
    outs = []
    for i, job in enumerate(jobs):
        X, wbits, wscale, group = job[:4]
        assert X.is_cuda and X.dtype == torch.float16 and X.dim() == 2 and X.stride(1) == 1
        M, K = X.shape
        N, ldw = wbits.shape
        if len(job) > 4:
            Y, D = job[4], job[5]
        else:
            Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
            D = torch.empty((M, N), dtype=torch.int32, device=X.device) if want_dots else None
        arr[i] = DecodeJobC(X.data_ptr(), M, K, _row_stride(X), wbits.data_ptr(), wscale.data_ptr(),
                            N, ldw, group, Y.data_ptr() if Y is not None else None,
                            _row_stride(Y) if Y is not None else N,
                            D.data_ptr() if D is not None else None,
                            _row_stride(D) if D is not None else N)
        outs.append((Y, D))
    return arr, outs


def bwta_linear_decode_batched(jobs, mode: int = TERNARY, thresh_ratio: float = 0.5,
                               want_dots: bool = False, flags: int = 0, status=None,
                               descriptors=None):
    """Several fused decode projections in one launch. `jobs` as decode_jobs();
    or pass `descriptors` = decode_jobs(...) built once (the outputs they name).
    Returns [(Y, dots or None)] per job."""
    lib = _L()
    arr, outs = descriptors if descriptors is not None else decode_jobs(jobs, want_dots)
    n = len(outs)
    _check("bwta_linear_decode_batched", lib.bwta_linear_decode_batched(
        arr, n, mode, thresh_ratio, flags, _ptr(status), _stream()))
    return outs


def bwta_attn_scores(q_mask, q_sign, q_scale, k_mask, k_sign, k_scale, BH: int, Lq: int, Lk: int,
                     D: int, want_int: bool = True, want_float: bool = True, out=None):
    """Ternary Q.K^T scores. Returns (S int32 [BH, Lq, Lk] or None, S fp32 or None)."""
    lib = _L()
    ld = q_mask.shape[-1]
    dev = q_mask.device
    if out is None:
        Si = torch.empty((BH, Lq, Lk), dtype=torch.int32, device=dev) if want_int else None
        Sf = torch.empty((BH, Lq, Lk), dtype=torch.float32, device=dev) if want_float else None
    else:
        Si, Sf = out
    _check("bwta_attn_scores", lib.bwta_attn_scores(
        _ptr(q_mask), _ptr(q_sign), _ptr(q_scale), _ptr(k_mask), _ptr(k_sign), _ptr(k_scale),
        BH, Lq, Lk, D, ld, _ptr(Si), _ptr(Sf), _stream()))
    return Si, Sf


def bwta_attn_softmax_ternarize(q_mask, q_sign, q_scale, k_mask, k_sign, k_scale, BH: int,
                                Lq: int, Lk: int, D: int, softmax_scale: float, out=None):
    """Ternary attention probabilities from ternary Q, K planes (scores never
    stored). Returns (p_mask, p_sign, p_scale): [BH*Lq, ld_words_for(Lk)] x2, [BH*Lq]."""
    lib = _L()
    ld = q_mask.shape[-1]
    ldp = ld_words_for(Lk)
    dev = q_mask.device
    if out is None:
        pm = torch.empty((BH * Lq, ldp), dtype=torch.int32, device=dev)
        ps = torch.empty((BH * Lq, ldp), dtype=torch.int32, device=dev)
        sc = torch.empty((BH * Lq,), dtype=torch.float32, device=dev)
    else:
        pm, ps, sc = out
    _check("bwta_attn_softmax_ternarize", lib.bwta_attn_softmax_ternarize(
        _ptr(q_mask), _ptr(q_sign), _ptr(q_scale), _ptr(k_mask), _ptr(k_sign), _ptr(k_scale),
        BH, Lq, Lk, D, ld, softmax_scale, _ptr(pm), _ptr(ps), pm.shape[1], _ptr(sc), _stream()))
    return pm, ps, sc


def bwta_attn_av(p_mask, p_sign, p_scale, vt_mask, vt_sign, vt_scale, BH: int, Lq: int, D: int,
                 Lk: int, want_int: bool = False, want_float: bool = True, out=None):
    """A . V with ternary probabilities and V^T planes. Returns (O int32 or None,
    O fp32 or None), each [BH, Lq, D]."""
    lib = _L()
    ld = p_mask.shape[-1]
    dev = p_mask.device
    if out is None:
        Oi = torch.empty((BH, Lq, D), dtype=torch.int32, device=dev) if want_int else None
        Of = torch.empty((BH, Lq, D), dtype=torch.float32, device=dev) if want_float else None
    else:
        Oi, Of = out
    _check("bwta_attn_av", lib.bwta_attn_av(
        _ptr(p_mask), _ptr(p_sign), _ptr(p_scale), _ptr(vt_mask), _ptr(vt_sign), _ptr(vt_scale),
        BH, Lq, D, Lk, ld, _ptr(Oi), _ptr(Of), _stream()))
    return Oi, Of


# ------------------------------------------------------------------ BiLLM
@dataclass
class BillmWeights:
    sign: torch.Tensor     # int32 [N, ldw]
    gmap: torch.Tensor     # int32 [N, ldw]
    res: torch.Tensor      # uint8 [N, K/block]
    sal: torch.Tensor      # uint8 [K/block, n_sal]
    bscale: torch.Tensor   # fp32 [N, K/block, 4]
    N: int
    K: int
    block: int = 128
    n_sal: int = 8

    @property
    def ldw(self) -> int:
        return self.sign.shape[1]

    def cstruct(self) -> BillmWeightsC:
        return BillmWeightsC(self.sign.data_ptr(), self.gmap.data_ptr(), self.res.data_ptr(),
                             self.sal.data_ptr() if self.sal.numel() else None,
                             self.bscale.data_ptr(), self.N, self.K, self.ldw, self.block,
                             self.n_sal)

    @staticmethod
    def empty(N: int, K: int, n_sal: int = 8, block: int = 128, device="cuda"):
        ld = ld_words_for(K)
        nb = K // block
        return BillmWeights(
            sign=torch.empty((N, ld), dtype=torch.int32, device=device),
            gmap=torch.empty((N, ld), dtype=torch.int32, device=device),
            res=torch.empty((N, nb), dtype=torch.uint8, device=device),
            sal=torch.empty((nb, n_sal), dtype=torch.uint8, device=device),
            bscale=torch.empty((N, nb, 4), dtype=torch.float32, device=device),
            N=N, K=K, block=block, n_sal=n_sal)


def billm_pack_weights(W: torch.Tensor, n_sal: int = 8, split=True, block: int = 128,
                       status=None) -> BillmWeights:
    """Latent fp32 W [N, K] (cuda) -> packed BiLLM weights, built on the GPU.
    split: False/0 no split, True/1 break-point 0.5*max|w|, 2 searched break-point."""
    lib = _L()
    assert W.is_cuda and W.dtype == torch.float32 and W.dim() == 2 and W.stride(1) == 1
    N, K = W.shape
    out = BillmWeights.empty(N, K, n_sal, block, W.device)
    cs = out.cstruct()
    _check("billm_pack_weights", lib.billm_pack_weights(
        _ptr(W), _row_stride(W), int(split), C.byref(cs), _ptr(status), _stream()))
    return out


def billm_gemm(X: torch.Tensor, Wq: BillmWeights, status=None, out=None) -> torch.Tensor:
    """fp16 X [M, K] x BiLLM weights -> Y fp32 [M, N]."""
    lib = _L()
    assert X.is_cuda and X.dtype == torch.float16 and X.dim() == 2 and X.stride(1) == 1
    M = X.shape[0]
    Y = out if out is not None else torch.empty((M, Wq.N), dtype=torch.float32, device=X.device)
    cs = Wq.cstruct()
    _check("billm_gemm", lib.billm_gemm(_ptr(X), M, _row_stride(X), C.byref(cs), _ptr(Y),
                                        _row_stride(Y), _ptr(status), _stream()))
    return Y


# ------------------------------------------------------------------ paged key-value cache
class KvCache:
    """One layer's pool of pages: k, v [num_pages, n_kv_heads, page_size, head_dim], fp16, or uint8
    (E4M3 bytes) with fp32 scales [num_pages, n_kv_heads, page_size]. Pages may be further apart than
    dense (a view of a larger buffer), the inner dimensions are dense. Keeps the tensors alive; their
    storage must stay where it is."""
    __slots__ = ("k", "v", "k_scale", "v_scale", "c", "ref", "device", "n_kv_heads", "head_dim", "page_size")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        e4m3 = k.dtype == torch.uint8
        assert k.is_cuda and k.dtype in (torch.float16, torch.uint8) and v.dtype == k.dtype
        assert k.dim() == 4 and v.shape == k.shape and v.device == k.device
        assert e4m3 == (k_scale is not None) == (v_scale is not None)
        P, H, ps, D = k.shape

        def stride(t, inner):
            """Distance of pages; the dimensions inside a page must be dense."""
            if t.is_contiguous():
                return inner
            step = 1
            for size, st in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
                assert size == 1 or st == step, "the dimensions inside a page must be dense"
                step *= size
            return t.stride(0) if t.shape[0] > 1 else inner

        rows = H * ps
        ld, ls = stride(k, rows * D), 0
        assert stride(v, rows * D) == ld
        if e4m3:
            for t in (k_scale, v_scale):
                assert t.dtype == torch.float32 and t.shape == k.shape[:3] and t.device == k.device
            ls = stride(k_scale, rows)
            assert stride(v_scale, rows) == ls
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.n_kv_heads, self.head_dim, self.page_size = k.device, H, D, ps
        self.c = KvCacheC(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if e4m3 else None,
                          v_scale.data_ptr() if e4m3 else None, P, ps, H, D, ld, ls,
                          KV_E4M3 if e4m3 else KV_F16)
        self.ref = C.byref(self.c)

    @staticmethod
    def empty(num_pages: int, page_size: int, n_kv_heads: int, head_dim: int, e4m3: bool = False,
              device="cuda"):
        shape = (num_pages, n_kv_heads, page_size, head_dim)
        kv = [torch.empty(shape, dtype=torch.uint8 if e4m3 else torch.float16, device=device)
              for _ in range(2)]
        sc = [torch.empty(shape[:3], dtype=torch.float32, device=device) if e4m3 else None
              for _ in range(2)]
        return KvCache(kv[0], kv[1], sc[0], sc[1])


class KvTable:
    """Which pages hold which sequence: pages int32 [n_slots, max_pages], kv_len int32 [n_slots],
    refcount int32 [num_pages] (needed by the page calls only). Keeps the tensors alive. The lengths mean
    pages of one size: with page_size given, every call on this table refuses another."""
    __slots__ = ("pages", "kv_len", "refcount", "c", "ref", "device", "page_size")

    def __init__(self, pages, kv_len, refcount=None, page_size=None):
        assert pages.is_cuda and pages.dtype == torch.int32 and pages.dim() == 2
        assert pages.shape[1] <= 1 or pages.stride(1) == 1
        assert kv_len.dtype == torch.int32 and kv_len.shape == pages.shape[:1]
        assert kv_len.is_contiguous() and kv_len.device == pages.device
        if refcount is not None:
            assert refcount.dtype == torch.int32 and refcount.dim() == 1
            assert refcount.is_contiguous() and refcount.device == pages.device
        self.pages, self.kv_len, self.refcount, self.device = pages, kv_len, refcount, pages.device
        self.page_size = page_size
        n, m = pages.shape
        self.c = KvTableC(pages.data_ptr(), max(pages.stride(0), m) if n > 1 else m, m, n,
                          kv_len.data_ptr(), refcount.data_ptr() if refcount is not None else None)
        assert n <= 1 or pages.stride(0) >= m
        self.ref = C.byref(self.c)

    @staticmethod
    def empty(n_slots: int, max_pages: int, num_pages: int, device="cuda", page_size=None):
        """A table without sequences over a pool of free pages."""
        return KvTable(torch.full((n_slots, max_pages), -1, dtype=torch.int32, device=device),
                       torch.zeros(n_slots, dtype=torch.int32, device=device),
                       torch.zeros(num_pages, dtype=torch.int32, device=device), page_size)

    def counts(self, page_size):
        """Whether the table's lengths are counted in pages of this size."""
        return self.page_size is None or self.page_size == page_size


class KvLayers:
    """The layers of a page call (KvCache each, one geometry) as C descriptors, built once."""
    __slots__ = ("caches", "c", "n", "num_pages", "page_size", "device")

    def __init__(self, caches):
        self.caches = list(caches)
        assert self.caches and all(x.device == self.caches[0].device for x in self.caches)
        self.c = (KvCacheC * len(self.caches))(*[x.c for x in self.caches])
        self.n = len(self.caches)
        self.num_pages, _, self.page_size, _ = self.caches[0].k.shape
        self.device = self.caches[0].device


def kv_layers(caches) -> KvLayers:
    """Descriptors for the page calls, from a KvCache or a list of them."""
    if isinstance(caches, KvLayers):
        return caches
    return KvLayers([caches] if isinstance(caches, KvCache) else caches)


_device_now = torch._C._cuda_getDevice
_stream_now = torch._C._cuda_getCurrentRawStream


def _kv_call(name, device, *args):
    """Call libbwta's `name` with these arguments and the current stream of `device`. The host's time
    is most of a small call's, so nothing here builds stream or device objects."""
    fn = getattr(_lib or _L(), name)
    dev = device.index
    if _device_now() == dev:
        rc = fn(*args, _stream_now(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream_now(dev))
    if rc != BWTA_OK:
        raise BwtaError(name, rc)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(name, *args):
    return getattr(load_library(), name)(*args)


def _ints(t, device):
    """Pointer of a dense int32 vector on `device` (or None)."""
    if t is None:
        return None
    assert t.dtype == torch.int32 and t.dim() == 1 and t.is_contiguous() and t.device == device
    return t.data_ptr()


def _status(t, device):
    if t is None:
        return None
    assert t.dtype == torch.int32 and t.numel() >= 1 and t.device == device
    return t.data_ptr()


def _kv_rows(t, width, device):
    """(pointer, row stride, rows) of rows of `width` values: [n, width] or [n, heads, dim]."""
    n = t.dim()
    assert t.device == device and n in (2, 3)
    if t.is_contiguous():
        rows = t.shape[0]
        assert (t.shape[1] * t.shape[2] if n == 3 else t.shape[1]) == width
        return t.data_ptr(), width, rows
    if n == 3:
        assert t.shape[2] <= 1 or t.stride(2) == 1
        assert t.shape[1] <= 1 or t.stride(1) == t.shape[2]
        assert t.shape[1] * t.shape[2] == width
    else:
        assert t.shape[1] == width and (width <= 1 or t.stride(1) == 1)
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else width), t.shape[0]


def bwta_kv_append(cache: KvCache, table: KvTable, k, v, slots=None, cu_q=None, status=None):
    """New tokens' keys and values, fp32 or fp16 [rows, n_kv_heads * head_dim] (or three dimensions),
    into the pages. Without cu_q one row for each slot (or for each of `slots`); with it rows
    cu_q[s] .. cu_q[s+1] belong to sequence s and end at its kv_len."""
    dev = cache.device
    assert table.device == dev and table.counts(cache.page_size)
    assert k.dtype == v.dtype and k.dtype in (torch.float16, torch.float32)
    width = cache.n_kv_heads * cache.head_dim
    kp, ldk, n = _kv_rows(k, width, dev)
    vp, ldv, nv = _kv_rows(v, width, dev)
    assert n == nv
    n_seq = _n_seq(table, slots, cu_q, n)
    _kv_call("bwta_kv_append", dev, cache.ref, table.ref, _ints(slots, dev), n_seq, _ints(cu_q, dev), n,
             kp, ldk, vp, ldv, int(k.dtype == torch.float32),
             _status(status, dev))


def _n_seq(table, slots, cu_q, rows):
    n = slots.shape[0] if slots is not None else (cu_q.shape[0] - 1 if cu_q is not None else rows)
    assert cu_q is None or cu_q.shape[0] == n + 1
    assert cu_q is not None or rows == n
    return n


def bwta_attn_decode_paged(q, cache: KvCache, table: KvTable, softmax_scale: float, window: int = 0,
                           sinks: int = 0, slots=None, workspace=None, status=None, out=None):
    """Attention of one new token of each sequence over its pages. q fp16 [n_seq, n_heads, head_dim]
    -> out, the same shape. workspace: uint8 of decode_workspace() bytes (allocated when not given)."""
    dev, D = cache.device, cache.head_dim
    assert q.dtype == torch.float16 and q.dim() == 3 and q.shape[2] == D
    assert table.device == dev and table.counts(cache.page_size)
    n, heads = q.shape[0], q.shape[1]
    qp, ldq, _ = _kv_rows(q, heads * D, dev)
    n_seq = _n_seq(table, slots, None, n)
    if out is None:
        out = torch.empty((n, heads, D), dtype=torch.float16, device=dev)
        op, ldo = out.data_ptr(), heads * D
    else:
        assert out.dtype == torch.float16 and out.shape == q.shape
        op, ldo, _ = _kv_rows(out, heads * D, dev)
    if workspace is None:
        workspace = decode_workspace(heads, cache)
    assert workspace.device == dev and workspace.is_contiguous()
    _kv_call("bwta_attn_decode_paged", dev, cache.ref, table.ref, _ints(slots, dev), n_seq, qp, ldq,
             heads, softmax_scale, window, sinks, op, ldo,
             workspace.data_ptr(), workspace.nbytes,
             _status(status, dev))
    return out


def decode_workspace(n_heads: int, cache: KvCache):
    """A workspace for bwta_attn_decode_paged; calls that may overlap in time need one each."""
    n = _workspace_bytes("bwta_attn_decode_workspace", n_heads, cache.n_kv_heads, cache.head_dim)
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def bwta_attn_prompt_paged(q, cu_q, cache: KvCache, table: KvTable, softmax_scale: float,
                           window: int = 0, sinks: int = 0, slots=None, status=None, out=None):
    """Attention of many new tokens of each sequence over its pages, which hold them already.
    q fp16 [rows, n_heads, head_dim], rows cu_q[s] .. cu_q[s+1] the newest of sequence s -> out, the
    same shape (rows past the last sequence are left as they are)."""
    dev, D = cache.device, cache.head_dim
    assert q.dtype == torch.float16 and q.dim() == 3 and q.shape[2] == D
    assert table.device == dev and table.counts(cache.page_size)
    n, heads = q.shape[0], q.shape[1]
    qp, ldq, _ = _kv_rows(q, heads * D, dev)
    n_seq = _n_seq(table, slots, cu_q, n)
    if out is None:
        out = torch.empty((n, heads, D), dtype=torch.float16, device=dev)
        op, ldo = out.data_ptr(), heads * D
    else:
        assert out.dtype == torch.float16 and out.shape == q.shape
        op, ldo, _ = _kv_rows(out, heads * D, dev)
    _kv_call("bwta_attn_prompt_paged", dev, cache.ref, table.ref, _ints(slots, dev), n_seq,
             _ints(cu_q, dev), n, qp, ldq, heads, softmax_scale, window,
             sinks, op, ldo, _status(status, dev))
    return out


def bwta_kv_reserve(table: KvTable, page_size: int, slots, n_new, status=None):
    """Room for n_new[i] more tokens in slot slots[i]; raises kv_len."""
    dev = table.device
    assert table.refcount is not None and slots.shape == n_new.shape and table.counts(page_size)
    _kv_call("bwta_kv_reserve", dev, table.ref, table.refcount.shape[0], page_size, _ints(slots, dev),
             _ints(n_new, dev), slots.shape[0], _status(status, dev))


def bwta_kv_free(table: KvTable, page_size: int, slots, status=None):
    """Give up the slots' pages."""
    dev = table.device
    assert table.refcount is not None and table.counts(page_size)
    _kv_call("bwta_kv_free", dev, table.ref, table.refcount.shape[0], page_size, _ints(slots, dev),
             slots.shape[0], _status(status, dev))


def pages_workspace(num_pages: int, n: int, device="cuda"):
    """A workspace for the page calls: num_pages of the pool (fork, compact) and n list entries."""
    return torch.empty(_workspace_bytes("bwta_kv_pages_workspace", num_pages, n), dtype=torch.uint8,
                       device=device)


def bwta_kv_fork(caches, table: KvTable, src, dst, workspace=None, status=None):
    """Make slot dst[i] a copy of slot src[i], in all layers: full pages shared, the rest copied."""
    l = kv_layers(caches)
    dev = l.device
    assert table.refcount is not None and table.refcount.shape[0] == l.num_pages
    assert src.shape == dst.shape and table.device == dev and table.counts(l.page_size)
    ws = pages_workspace(l.num_pages, src.shape[0], dev) if workspace is None else workspace
    assert ws.device == dev and ws.is_contiguous()
    _kv_call("bwta_kv_fork", dev, l.c, l.n, table.ref, _ints(src, dev), _ints(dst, dev), src.shape[0],
             ws.data_ptr(), ws.nbytes, _status(status, dev))


def bwta_kv_compact(caches, table: KvTable, workspace=None, status=None, out=None):
    """Move the pages in use to the front of the pool, in all layers. Returns int32 [1]: how many."""
    l = kv_layers(caches)
    dev = l.device
    assert table.refcount is not None and table.refcount.shape[0] == l.num_pages
    assert table.device == dev and table.counts(l.page_size)
    ws = pages_workspace(l.num_pages, 0, dev) if workspace is None else workspace
    assert ws.device == dev and ws.is_contiguous()
    if out is None:
        out = torch.empty(1, dtype=torch.int32, device=dev)
    _kv_call("bwta_kv_compact", dev, l.c, l.n, table.ref, _ints(out, dev), ws.data_ptr(), ws.nbytes,
             _status(status, dev))
    return out


def bwta_kv_copy_pages(src_caches, dst_caches, src_pages, dst_pages, workspace=None, status=None):
    """Copy page src_pages[i] of src to page dst_pages[i] of dst, in all layers."""
    a, b = kv_layers(src_caches), kv_layers(dst_caches)
    dev = a.device
    assert b.device == dev and a.n == b.n and src_pages.shape == dst_pages.shape
    n = src_pages.shape[0]
    ws = pages_workspace(0, n, dev) if workspace is None else workspace
    assert ws.device == dev and ws.is_contiguous()
    _kv_call("bwta_kv_copy_pages", dev, a.c, b.c, a.n, _ints(src_pages, dev), _ints(dst_pages, dev), n,
             ws.data_ptr(), ws.nbytes, _status(status, dev))


# ------------------------------------------------------------------ helpers
def as_u32(t: torch.Tensor):
    """A bit-plane tensor (int32 on any device) as a numpy uint32 array."""
    return t.detach().cpu().numpy().view("uint32")


def half_from_numpy(x, device="cuda") -> torch.Tensor:
    return torch.from_numpy(x).to(device)
