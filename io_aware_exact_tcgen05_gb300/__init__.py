"""GB300-native exact tiled attention: thin Python binding over libfa.so.

Every function here only marshals arguments (device pointers, sizes, the
current CUDA stream) into the C ABI declared in ``include/fa.h``; all of the
attention arithmetic runs in the library's sm_103a kernels.  PyTorch is used
only to allocate device memory and to provide streams.  There is no CPU or
PyTorch fallback: if ``libfa.so`` is missing or fails to load, every call
raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_WORKSPACE = 3
FA_ERR_CUDA = 4
FA_ERR_TIMEOUT = 5

EXPORTED = ("fa_fwd", "fa_bwd", "fa_bwd_workspace_size", "fa_decode", "fa_decode_workspace_size",
            "fa_decode_noalloc", "fa_fwd_masked", "fa_bwd_masked", "fa_fwd_varlen",
            "fa_bwd_varlen", "fa_fwd_dropout", "fa_bwd_dropout", "fa_key_mask_words",
            "fa_pack_key_mask", "fa_fwd_fp8", "fa_kv_assign", "fa_kv_write_fp8", "fa_kv_read_fp8",
            "fa_select_blocks", "fa_select_blocks_workspace_size", "fa_decode_paged_fp8",
            "fa_decode_paged_fp8_workspace_size", "fa_qk_norm_rope", "fa_qk_norm_rope_bwd",
            "fa_qk_norm_rope_bwd_workspace_size", "fa_row_bounds", "fa_mask_plan",
            "fa_mask_plan_size", "fa_fwd_scored", "fa_fwd_scored_workspace_size", "fa_bwd_scored",
            "fa_bwd_scored_workspace_size", "fa_decode_scored", "fa_decode_scored_workspace_size", "fa_device_status", "fa_selftest_wait_timeout",
            "fa_profile_next_launch", "fa_status_string", "fa_last_error_detail", "fa_version")

_lib = None


class _Heads(ctypes.Structure):
    """fa_heads of include/fa.h: a strided view [B, S, H, d]."""
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_longlong),
                ("stride_t", ctypes.c_longlong), ("stride_h", ctypes.c_longlong)]


class FAError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: status {status}: {detail}")
        self.status = status


def load_library(path: str = LIB_PATH):
    """Load libfa.so (build it first with ``io_aware_exact_tcgen05_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libfa.so not found at {path}: run __graft_entry__.build() first")
    lib = ctypes.CDLL(path)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, F, P, P, P]
    lib.fa_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P, P, P, Z, P]
    lib.fa_decode.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, P, Z, P]
    lib.fa_decode_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, P]
    lib.fa_fwd_masked.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, F, P, P, P, P]
    lib.fa_bwd_masked.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P, P, P, P, Z,
                                  P]
    lib.fa_fwd_varlen.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, P, P]
    lib.fa_bwd_varlen.argtypes = [P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, P,
                                  P, Z, P]
    U64, U32 = ctypes.c_ulonglong, ctypes.c_uint
    lib.fa_fwd_dropout.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, F, P, P, P, F, U64, U32, P]
    lib.fa_bwd_dropout.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P, P, P, F,
                                   U64, U32, P, Z, P]
    lib.fa_fwd_dropout.restype = I
    lib.fa_bwd_dropout.restype = I
    lib.fa_fwd_fp8.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, F, F, F, F, P, P, P]
    lib.fa_fwd_fp8.restype = I
    lib.fa_key_mask_words.argtypes = [I]
    lib.fa_key_mask_words.restype = Z
    lib.fa_pack_key_mask.argtypes = [P, P, I, I, P]
    for f in (lib.fa_fwd_masked, lib.fa_bwd_masked, lib.fa_fwd_varlen, lib.fa_bwd_varlen,
              lib.fa_pack_key_mask):
        f.restype = I
    lib.fa_decode_noalloc.restype = I
    lib.fa_bwd_workspace_size.argtypes = [I, I, I, I]
    lib.fa_bwd_workspace_size.restype = Z
    lib.fa_decode_workspace_size.argtypes = [I, I, I, I]
    lib.fa_decode_workspace_size.restype = Z
    lib.fa_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint), I]
    for f in (lib.fa_fwd, lib.fa_bwd, lib.fa_decode, lib.fa_device_status):
        f.restype = I
    lib.fa_selftest_wait_timeout.argtypes = [P, P]
    lib.fa_selftest_wait_timeout.restype = I
    lib.fa_profile_next_launch.argtypes = [P, P]
    lib.fa_profile_next_launch.restype = I
    L = ctypes.c_longlong
    lib.fa_kv_assign.argtypes = [P, P, I, I, P, I, P, I, P, I, P, P, P, P, P]
    lib.fa_kv_write_fp8.argtypes = [P, P, L, L, L, L, P, I, P, P, P, P, P, I, I, I, I, P]
    lib.fa_kv_read_fp8.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P]
    lib.fa_select_blocks.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, I, P, Z, P]
    lib.fa_decode_paged_fp8.argtypes = [P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I,
                                        F, P, Z, P]
    for f in (lib.fa_kv_assign, lib.fa_kv_write_fp8, lib.fa_kv_read_fp8, lib.fa_select_blocks,
              lib.fa_decode_paged_fp8):
        f.restype = I
    lib.fa_select_blocks_workspace_size.argtypes = [I, I, I]
    lib.fa_select_blocks_workspace_size.restype = Z
    lib.fa_decode_paged_fp8_workspace_size.argtypes = [I, I, I, I, I]
    lib.fa_decode_paged_fp8_workspace_size.restype = Z
    H = ctypes.POINTER(_Heads)
    lib.fa_qk_norm_rope.argtypes = [H, H, H, P, P, P, P, I, P, P, F, F, P, I, P, P, I, I, I, I, I, I,
                                    I, P]
    lib.fa_qk_norm_rope_bwd.argtypes = [H, H, P, P, P, H, H, H, P, P, P, P, F, F, P, I, P, P, I, I, I,
                                        I, I, I, I, P, Z, P]
    lib.fa_row_bounds.argtypes = [P, P, I, P, P, I, I, I, I, I, P]
    lib.fa_mask_plan.argtypes = [P, P, I, I, I, P, Z, P]
    lib.fa_fwd_scored.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, F, F, P, P, Z, P, Z, P]
    lib.fa_bwd_scored.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, F, P, P, Z, P, Z, P]
    lib.fa_decode_scored.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F, F, P, I, P, Z, P]
    for f in (lib.fa_qk_norm_rope, lib.fa_qk_norm_rope_bwd, lib.fa_row_bounds, lib.fa_mask_plan,
              lib.fa_fwd_scored, lib.fa_bwd_scored, lib.fa_decode_scored):
        f.restype = I
    lib.fa_qk_norm_rope_bwd_workspace_size.argtypes = [I]
    lib.fa_mask_plan_size.argtypes = [I, I, I]
    lib.fa_fwd_scored_workspace_size.argtypes = [I, I, I, I, I, I]
    lib.fa_bwd_scored_workspace_size.argtypes = [I, I, I, I, I, I]
    lib.fa_decode_scored_workspace_size.argtypes = [I, I, I, I, I, I]
    for f in (lib.fa_qk_norm_rope_bwd_workspace_size, lib.fa_mask_plan_size,
              lib.fa_fwd_scored_workspace_size, lib.fa_bwd_scored_workspace_size,
              lib.fa_decode_scored_workspace_size):
        f.restype = Z
    lib.fa_status_string.argtypes = [I]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_last_error_detail.restype = ctypes.c_char_p
    lib.fa_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != FA_OK:
        detail = _lib.fa_last_error_detail().decode()
        raise FAError(status, where, detail or _lib.fa_status_string(status).decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    # the raw handle: building a torch.cuda.Stream costs some 10 us a call
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _need(t, name, dtype, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


def fa_key_mask_words(Sk: int) -> int:
    return int(load_library().fa_key_mask_words(Sk))


def fa_pack_key_mask(mask, stream=None):
    """Visibility bit words [rows, fa_key_mask_words(Sk)] (int32 storage of the
    uint32 words) from a bool/uint8 CUDA mask [rows, Sk], via fa_pack_key_mask."""
    lib = load_library()
    if not isinstance(mask, torch.Tensor) or not mask.is_cuda:
        raise TypeError("mask must be a CUDA tensor")
    if mask.dtype not in (torch.bool, torch.uint8) or not mask.is_contiguous() or mask.dim() != 2:
        raise ValueError("mask must be a contiguous 2-D bool or uint8 tensor")
    rows, Sk = mask.shape
    bits = torch.empty(rows, fa_key_mask_words(Sk), dtype=torch.int32, device=mask.device)
    _check(lib.fa_pack_key_mask(_ptr(mask), _ptr(bits), rows, Sk, _stream(stream)),
           "fa_pack_key_mask")
    return bits


def _mask_bits(key_mask, rows, Sk, stream):
    """Bit words for a key mask given as bools [rows, Sk] (packed on the
    device) or as bit words already; None when there is no mask."""
    if key_mask is None:
        return None
    if key_mask.dtype in (torch.bool, torch.uint8):
        if tuple(key_mask.shape) != (rows, Sk):
            raise ValueError(f"key_mask must be [{rows}, {Sk}], got {tuple(key_mask.shape)}")
        return fa_pack_key_mask(key_mask.contiguous(), stream)
    _need(key_mask, "key_mask bits", torch.int32, 2)
    if tuple(key_mask.shape) != (rows, fa_key_mask_words(Sk)):
        raise ValueError("key_mask bit words have the wrong shape")
    return key_mask


def fa_fwd(q, k, v, causal: bool, scale: float, k_start=None, k_end=None, o=None, lse=None,
           stream=None, key_mask=None, dropout_p: float = 0.0, seed: int = 0, offset: int = 0):
    """O, LSE = attention(q, k, v) via the library's fa_fwd (see include/fa.h).
    q [B,Hq,Sq,d], k/v [B,Hkv,Sk,d] bf16 CUDA tensors; k_start/k_end optional
    int32 [B] CUDA tensors; key_mask optional [B, Sk] bool CUDA tensor (or its
    fa_pack_key_mask words), giving fa_fwd_masked.  dropout_p > 0 (taken as
    float32) gives fa_fwd_dropout with the given seed and offset.
    Returns (o, lse)."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 4)
    B, Hq, Sq, d = q.shape
    _, Hkv, Sk, _ = k.shape
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hq, Sq, dtype=torch.float32, device=q.device)
    for t, n in ((k_start, "k_start"), (k_end, "k_end")):
        if t is not None:
            _need(t, n, torch.int32, 1)
    bits = _mask_bits(key_mask, B, Sk, stream)
    if dropout_p > 0.0:
        st = lib.fa_fwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Sq,
                                Sk, d, int(bool(causal)), float(scale), _ptr(k_start),
                                _ptr(k_end), _ptr(bits), float(dropout_p), int(seed),
                                int(offset), _stream(stream))
        _check(st, "fa_fwd_dropout")
    elif bits is None:
        st = lib.fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Sq, Sk, d,
                        int(bool(causal)), float(scale), _ptr(k_start), _ptr(k_end),
                        _stream(stream))
        _check(st, "fa_fwd")
    else:
        st = lib.fa_fwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Sq, Sk,
                               d, int(bool(causal)), float(scale), _ptr(k_start), _ptr(k_end),
                               _ptr(bits), _stream(stream))
        _check(st, "fa_fwd_masked")
    return o, lse


def _need8(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    f8 = getattr(torch, "float8_e4m3fn", None)
    if t.dtype not in tuple(x for x in (f8, torch.uint8) if x is not None):
        raise TypeError(f"{name} must hold e4m3 bytes (float8_e4m3fn or uint8), got {t.dtype}")
    if not t.is_contiguous() or t.dim() != 4:
        raise ValueError(f"{name} must be a contiguous 4-D tensor")


def fa_fwd_fp8(q8, k8, vt8, causal: bool, scale: float, q_descale: float, k_descale: float,
               v_descale: float, k_start=None, k_end=None, o=None, lse=None, stream=None):
    """FP8 forward via fa_fwd_fp8: q8 [B,Hq,Sq,128], k8 [B,Hkv,Sk,128] and
    vt8 [B,Hkv,128,Sk] (V transposed) e4m3 CUDA tensors with per-tensor
    descale factors.  Returns (o bf16 [B,Hq,Sq,128], lse [B,Hq,Sq])."""
    lib = load_library()
    for t, n in ((q8, "q8"), (k8, "k8"), (vt8, "vt8")):
        _need8(t, n)
    B, Hq, Sq, d = q8.shape
    _, Hkv, Sk, _ = k8.shape
    if tuple(vt8.shape) != (B, Hkv, d, Sk):
        raise ValueError(f"vt8 must be [B, Hkv, d, Sk] = {(B, Hkv, d, Sk)}")
    o = torch.empty(B, Hq, Sq, d, dtype=torch.bfloat16, device=q8.device) if o is None else o
    lse = torch.empty(B, Hq, Sq, dtype=torch.float32, device=q8.device) if lse is None else lse
    st = lib.fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(vt8), _ptr(o), _ptr(lse), B, Hq, Hkv, Sq, Sk, d,
                        int(bool(causal)), float(scale), float(q_descale), float(k_descale),
                        float(v_descale), _ptr(k_start), _ptr(k_end), _stream(stream))
    _check(st, "fa_fwd_fp8")
    return o, lse


def fa_bwd_workspace_size(B, Hq, Sq, d) -> int:
    return int(load_library().fa_bwd_workspace_size(B, Hq, Sq, d))


def fa_bwd(q, k, v, o, dout, lse, causal: bool, scale: float, k_start=None, k_end=None,
           dq=None, dk=None, dv=None, workspace=None, stream=None, key_mask=None,
           dropout_p: float = 0.0, seed: int = 0, offset: int = 0):
    """dQ, dK, dV by recomputation via the library's fa_bwd (fa_bwd_masked
    when key_mask is given, fa_bwd_dropout when dropout_p > 0; mask and
    dropout arguments must be the forward's).  Returns (dq, dk, dv)."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _need(t, n, torch.bfloat16, 4)
    _need(lse, "lse", torch.float32, 3)
    B, Hq, Sq, d = q.shape
    _, Hkv, Sk, _ = k.shape
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    nbytes = fa_bwd_workspace_size(B, Hq, Sq, d)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    bits = _mask_bits(key_mask, B, Sk, stream)
    if dropout_p > 0.0:
        st = lib.fa_bwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                _ptr(dq), _ptr(dk), _ptr(dv), B, Hq, Hkv, Sq, Sk, d,
                                int(bool(causal)), float(scale), _ptr(k_start), _ptr(k_end),
                                _ptr(bits), float(dropout_p), int(seed), int(offset),
                                _ptr(workspace), workspace.numel(), _stream(stream))
        _check(st, "fa_bwd_dropout")
    elif bits is None:
        st = lib.fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                        _ptr(dk), _ptr(dv), B, Hq, Hkv, Sq, Sk, d, int(bool(causal)),
                        float(scale), _ptr(k_start), _ptr(k_end), _ptr(workspace),
                        workspace.numel(), _stream(stream))
        _check(st, "fa_bwd")
    else:
        st = lib.fa_bwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                               _ptr(dq), _ptr(dk), _ptr(dv), B, Hq, Hkv, Sq, Sk, d,
                               int(bool(causal)), float(scale), _ptr(k_start), _ptr(k_end),
                               _ptr(bits), _ptr(workspace), workspace.numel(), _stream(stream))
        _check(st, "fa_bwd_masked")
    return dq, dk, dv


def _varlen_args(q, k, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k):
    for t, n in ((cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_k, "cu_seqlens_k")):
        _need(t, n, torch.int32, 1)
    if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 2:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both hold nseq + 1 >= 2 offsets")
    Hq, total_q, d = q.shape
    Hkv, total_k, _ = k.shape
    return cu_seqlens_q.numel() - 1, Hq, Hkv, total_q, total_k, d


def fa_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                  causal: bool, scale: float, key_mask=None, o=None, lse=None, stream=None):
    """Packed ragged forward via fa_fwd_varlen: q [Hq,total_q,d], k/v
    [Hkv,total_k,d] bf16; cu_seqlens_* int32 [nseq+1] CUDA offsets; key_mask
    optional [total_k] bools over the packed keys.  Returns (o, lse [Hq,total_q])."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 3)
    nseq, Hq, Hkv, total_q, total_k, d = _varlen_args(q, k, cu_seqlens_q, cu_seqlens_k,
                                                      max_seqlen_q, max_seqlen_k)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty(Hq, total_q, dtype=torch.float32, device=q.device) if lse is None else lse
    bits = _mask_bits(None if key_mask is None else key_mask.reshape(1, -1), 1, total_k, stream)
    st = lib.fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens_q),
                           _ptr(cu_seqlens_k), nseq, int(max_seqlen_q), int(max_seqlen_k),
                           total_q, total_k, Hq, Hkv, d, int(bool(causal)), float(scale),
                           _ptr(bits), _stream(stream))
    _check(st, "fa_fwd_varlen")
    return o, lse


def fa_bwd_varlen(q, k, v, o, dout, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                  max_seqlen_k: int, causal: bool, scale: float, key_mask=None, dq=None,
                  dk=None, dv=None, workspace=None, stream=None):
    """Packed ragged backward via fa_bwd_varlen (layout of fa_fwd_varlen).
    Returns (dq [Hq,total_q,d], dk, dv [Hkv,total_k,d])."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _need(t, n, torch.bfloat16, 3)
    _need(lse, "lse", torch.float32, 2)
    nseq, Hq, Hkv, total_q, total_k, d = _varlen_args(q, k, cu_seqlens_q, cu_seqlens_k,
                                                      max_seqlen_q, max_seqlen_k)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = torch.empty(fa_bwd_workspace_size(1, Hq, total_q, d), dtype=torch.uint8,
                                device=q.device)
    bits = _mask_bits(None if key_mask is None else key_mask.reshape(1, -1), 1, total_k, stream)
    st = lib.fa_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                           _ptr(dk), _ptr(dv), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), nseq,
                           int(max_seqlen_q), int(max_seqlen_k), total_q, total_k, Hq, Hkv, d,
                           int(bool(causal)), float(scale), _ptr(bits), _ptr(workspace),
                           workspace.numel(), _stream(stream))
    _check(st, "fa_bwd_varlen")
    return dq, dk, dv


def fa_decode_workspace_size(B, Hq, Sk_max, d) -> int:
    return int(load_library().fa_decode_workspace_size(B, Hq, Sk_max, d))


def fa_decode(q, k_cache, v_cache, seqlens_k, scale: float, o=None, lse=None, workspace=None,
              stream=None):
    """Single-query decode over a padded cache via the library's fa_decode.
    q [B,Hq,1,d], k_cache/v_cache [B,Hkv,Sk_max,d], seqlens_k int32 [B] (CUDA).
    Returns (o [B,Hq,1,d], lse [B,Hq])."""
    lib = load_library()
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.bfloat16, 4)
    _need(seqlens_k, "seqlens_k", torch.int32, 1)
    B, Hq, _, d = q.shape
    _, Hkv, Sk_max, _ = k_cache.shape
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device) if lse is None else lse
    nbytes = fa_decode_workspace_size(B, Hq, Sk_max, d)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    st = lib.fa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse),
                       _ptr(seqlens_k), B, Hq, Hkv, Sk_max, d, float(scale), _ptr(workspace),
                       workspace.numel(), _stream(stream))
    _check(st, "fa_decode")
    return o, lse


DECODE_NOALLOC_MAX_SCRATCH_BYTES = 64 << 20


def fa_decode_noalloc(q, k_cache, v_cache, seqlens_k, scale: float, o=None, lse=None,
                      stream=None):
    """fa_decode without a caller workspace: the library uses its built-in
    64 MiB scratch array instead (see include/fa.h).  For callers that cannot
    allocate device scratch; outputs may still be passed in.  Calls that can
    overlap on the GPU share that scratch and race."""
    lib = load_library()
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.bfloat16, 4)
    _need(seqlens_k, "seqlens_k", torch.int32, 1)
    B, Hq, _, d = q.shape
    _, Hkv, Sk_max, _ = k_cache.shape
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device) if lse is None else lse
    st = lib.fa_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse),
                               _ptr(seqlens_k), B, Hq, Hkv, Sk_max, d, float(scale),
                               _stream(stream))
    _check(st, "fa_decode_noalloc")
    return o, lse


# --------------------------------------------------- paged 8-bit KV cache --
#
# A decode step calls these with a microsecond or two of kernel time each, so a
# tensor's checks are one expression; what is wrong is worked out only then.

_BF16, _F32, _I32, _I64, _I8 = (torch.bfloat16, torch.float32, torch.int32, torch.int64,
                                torch.int8)
_U8 = torch.uint8
_F8 = getattr(torch, "float8_e4m3fn", torch.uint8)


def _device():
    """The current device's index; -2 (no tensor's) where there is no GPU."""
    try:
        return torch._C._cuda_getDevice()
    except RuntimeError:
        return -2


def _refuse(t, name, dtype, shape, dev):
    """Raise for the first thing about t that is not as the call needs it."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"tensors must be on the current device (cuda:{dev}), {name} is on "
                         f"{t.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _have(t, name, dtype, shape, dev):
    """t is a contiguous `dtype` tensor of that shape on the current device."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.get_device() == dev
            and t.shape == shape and t.is_contiguous()):
        _refuse(t, name, dtype, shape, dev)


def _dims(t, name, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if len(shape) != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    if max(shape) > 0x7fffffff:  # cut to its low 32 bits on the way
        raise ValueError(f"a size of {name} ({max(shape)}) does not fit 32 bits")
    return shape


def _int(x, name):
    """x as a C int: a larger value would be cut to its low 32 bits on the way."""
    x = int(x)
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError(f"{name} ({x}) does not fit 32 bits")
    return x


@functools.lru_cache(None)
def _cuda(dev):
    """Device `dev` as an object: torch.empty takes 1.4 us longer with the number."""
    return torch.device("cuda", dev)


def _new(shape, dtype, dev, stream):
    """An output or workspace for a call on `stream`, from that stream's memory: what
    the current stream's allocations are cut from may still be in use by its
    pending work.  The current stream may go on to use it (after a wait)."""
    here = None if stream is None else torch.cuda.current_stream()
    if stream == here:
        return torch.empty(shape, dtype=dtype, device=_cuda(dev))
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=_cuda(dev))
    t.record_stream(here)
    return t


def _out(t, name, shape, dtype, dev, stream):
    if t is None:
        return _new(shape, dtype, dev, stream)
    _have(t, name, dtype, shape, dev)
    return t


def _workspace(ws, nbytes, dev, stream):
    if ws is None:
        return _new((max(nbytes, 16),), _U8, dev, stream)
    if not (isinstance(ws, torch.Tensor) and ws.get_device() == dev and ws.is_contiguous()):
        raise TypeError("workspace must be a contiguous CUDA tensor on the current device")
    return ws


def _need_cache(k_cache, v_cache, k_scale, v_scale, dev):
    """Shape (num_pages, Hkv, page_size, d) of a cache, checked."""
    shape = _dims(k_cache, "k_cache", 4)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if isinstance(t, torch.Tensor) and t.dtype not in (_U8, _F8):
            raise TypeError(f"{n} must hold e4m3 bytes (float8_e4m3fn or uint8), got {t.dtype}")
        _have(t, n, getattr(t, "dtype", _U8), shape, dev)
    _have(k_scale, "k_scale", _F32, shape[:2], dev)
    _have(v_scale, "v_scale", _F32, shape[:2], dev)
    return shape


def fa_kv_assign(seqlens, newlens, page_size: int, block_table, free_pages, total_new: int,
                 slot_map=None, cu_new=None, seqlens_out=None, cu_seqlens_k=None, n_used=None,
                 stream=None):
    """Pages and slots for newlens[b] new tokens of every request (fa_kv_assign):
    block_table int32 [B,max_blocks] gets the entries of the new blocks, taken
    off the front of free_pages int32 [n_free].  Returns (slot_map int64
    [total_new], cu_new int32 [B+1], seqlens_out int32 [B], cu_seqlens_k int32
    [B+1], n_used int32 [1])."""
    lib, dev = load_library(), _device()
    B, max_blocks = _dims(block_table, "block_table", 2)
    _have(block_table, "block_table", _I32, (B, max_blocks), dev)
    _have(seqlens, "seqlens", _I32, (B,), dev)
    _have(newlens, "newlens", _I32, (B,), dev)
    n_free, = _dims(free_pages, "free_pages", 1)
    _have(free_pages, "free_pages", _I32, (n_free,), dev)
    total_new, page_size = _int(total_new, "total_new"), _int(page_size, "page_size")
    slot_map = _out(slot_map, "slot_map", (total_new,), _I64, dev, stream)
    cu_new = _out(cu_new, "cu_new", (B + 1,), _I32, dev, stream)
    seqlens_out = _out(seqlens_out, "seqlens_out", (B,), _I32, dev, stream)
    cu_seqlens_k = _out(cu_seqlens_k, "cu_seqlens_k", (B + 1,), _I32, dev, stream)
    n_used = _out(n_used, "n_used", (1,), _I32, dev, stream)
    st = lib.fa_kv_assign(seqlens.data_ptr(), newlens.data_ptr(), B, page_size,
                          block_table.data_ptr(), max_blocks, free_pages.data_ptr(), n_free,
                          slot_map.data_ptr(), total_new, cu_new.data_ptr(),
                          seqlens_out.data_ptr(), cu_seqlens_k.data_ptr(), n_used.data_ptr(),
                          _stream(stream))
    _check(st, "fa_kv_assign")
    return slot_map, cu_new, seqlens_out, cu_seqlens_k, n_used


def fa_kv_write_fp8(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, k_bounds=None,
                    stream=None):
    """Quantise new keys and values into the cache, in place (fa_kv_write_fp8).
    k, v bf16 [Hkv, n, d], or any view of that shape whose channels are
    contiguous and whose other strides are multiples of 8 (a token-major
    projection output, transposed); slot_map int64 [n]; k_cache/v_cache e4m3
    [num_pages,Hkv,page_size,d]; k_scale/v_scale fp32 [num_pages,Hkv]; k_bounds
    int8 [num_pages,Hkv,2,d] when blocks are to be selected."""
    lib, dev = load_library(), _device()
    num_pages, Hkv, ps, d = _need_cache(k_cache, v_cache, k_scale, v_scale, dev)
    n, = _dims(slot_map, "slot_map", 1)
    _have(slot_map, "slot_map", _I64, (_int(n, "the number of tokens"),), dev)
    strides = []
    for t, name in ((k, "k"), (v, "v")):
        if not (isinstance(t, torch.Tensor) and t.dtype == _BF16 and t.get_device() == dev
                and t.shape == (Hkv, n, d)):
            _refuse(t, name, _BF16, (Hkv, n, d), dev)
        st_h, st_t, st_c = t.stride()
        if n > 0 and st_c != 1:
            raise ValueError(f"{name} must have contiguous channels")
        # a dimension of one element is never stepped over: its stride does not matter
        strides += [st_h if Hkv > 1 else 0, st_t if n > 1 else 0]
    if k_bounds is not None:
        _have(k_bounds, "k_bounds", _I8, (num_pages, Hkv, 2, d), dev)
    st = lib.fa_kv_write_fp8(k.data_ptr(), v.data_ptr(), *strides, slot_map.data_ptr(), n,
                             k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                             v_scale.data_ptr(), _ptr(k_bounds), num_pages, Hkv, ps, d,
                             _stream(stream))
    _check(st, "fa_kv_write_fp8")


def fa_kv_read_fp8(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens_k, total_k: int,
                   k=None, v=None, stream=None):
    """Cached keys and values as packed bf16 [Hkv,total_k,d] (fa_kv_read_fp8), the
    layout of fa_fwd_varlen; cu_seqlens_k int32 [nseq+1].  Rows of no sequence
    are left as they were (unset in new outputs).  Returns (k, v)."""
    lib, dev = load_library(), _device()
    num_pages, Hkv, ps, d = _need_cache(k_cache, v_cache, k_scale, v_scale, dev)
    nseq, max_blocks = _dims(block_table, "block_table", 2)
    _have(block_table, "block_table", _I32, (nseq, max_blocks), dev)
    _have(cu_seqlens_k, "cu_seqlens_k", _I32, (nseq + 1,), dev)
    total_k = _int(total_k, "total_k")
    k = _out(k, "k", (Hkv, total_k, d), _BF16, dev, stream)
    v = _out(v, "v", (Hkv, total_k, d), _BF16, dev, stream)
    st = lib.fa_kv_read_fp8(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                            v_scale.data_ptr(), block_table.data_ptr(), cu_seqlens_k.data_ptr(),
                            k.data_ptr(), v.data_ptr(), nseq, max_blocks, num_pages, total_k, Hkv,
                            ps, d, _stream(stream))
    _check(st, "fa_kv_read_fp8")
    return k, v


def fa_select_blocks_workspace_size(B, Hkv, max_blocks) -> int:
    return int(load_library().fa_select_blocks_workspace_size(
        _int(B, "B"), _int(Hkv, "Hkv"), _int(max_blocks, "max_blocks")))


def fa_select_blocks(q, k_bounds, k_scale, block_table, seqlens_k, page_size: int, k_blocks: int,
                     n_first: int = 1, n_last: int = 1, sel=None, n_sel=None, workspace=None,
                     stream=None):
    """The k_blocks blocks of each request and KV head with the largest bound on
    their scores (fa_select_blocks), always with the first n_first and last
    n_last.  q bf16 [B,Hq,Sq,d].  Returns (sel int32 [B,Hkv,k_blocks] ascending,
    filled up with -1, n_sel int32 [B,Hkv])."""
    lib, dev = load_library(), _device()
    B, Hq, Sq, d = _dims(q, "q", 4)
    num_pages, Hkv = _dims(k_scale, "k_scale", 2)
    max_blocks = _dims(block_table, "block_table", 2)[1]
    _have(q, "q", _BF16, (B, Hq, Sq, d), dev)
    _have(k_scale, "k_scale", _F32, (num_pages, Hkv), dev)
    _have(k_bounds, "k_bounds", _I8, (num_pages, Hkv, 2, d), dev)
    _have(block_table, "block_table", _I32, (B, max_blocks), dev)
    _have(seqlens_k, "seqlens_k", _I32, (B,), dev)
    k_blocks, page_size = _int(k_blocks, "k_blocks"), _int(page_size, "page_size")
    n_first, n_last = _int(n_first, "n_first"), _int(n_last, "n_last")
    sel = _out(sel, "sel", (B, Hkv, max(k_blocks, 0)), _I32, dev, stream)
    n_sel = _out(n_sel, "n_sel", (B, Hkv), _I32, dev, stream)
    workspace = _workspace(workspace, lib.fa_select_blocks_workspace_size(B, Hkv, max_blocks), dev,
                           stream)
    st = lib.fa_select_blocks(q.data_ptr(), k_bounds.data_ptr(), k_scale.data_ptr(),
                              block_table.data_ptr(), seqlens_k.data_ptr(), sel.data_ptr(),
                              n_sel.data_ptr(), B, Hq, Hkv, Sq, num_pages, max_blocks,
                              page_size, d, k_blocks, n_first, n_last,
                              workspace.data_ptr(), workspace.nbytes, _stream(stream))
    _check(st, "fa_select_blocks")
    return sel, n_sel


def fa_decode_paged_fp8_workspace_size(B, Hq, Hkv, Sq, d) -> int:
    return int(load_library().fa_decode_paged_fp8_workspace_size(
        _int(B, "B"), _int(Hq, "Hq"), _int(Hkv, "Hkv"), _int(Sq, "Sq"), _int(d, "d")))


def fa_decode_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k,
                        scale: float, sel=None, n_sel=None, o=None, lse=None, workspace=None,
                        stream=None):
    """Attention of the last Sq tokens of each request over the paged 8-bit cache
    (fa_decode_paged_fp8).  q bf16 [B,Hq,Sq,d]; seqlens_k int32 [B] counts the Sq
    tokens too; sel/n_sel (fa_select_blocks) restrict each KV head to the listed
    blocks.  Returns (o bf16 [B,Hq,Sq,d], lse fp32 [B,Hq,Sq])."""
    lib, dev = load_library(), _device()
    B, Hq, Sq, d = shape = _dims(q, "q", 4)
    _have(q, "q", _BF16, shape, dev)
    num_pages, Hkv, ps, dc = _need_cache(k_cache, v_cache, k_scale, v_scale, dev)
    if dc != d:
        raise ValueError(f"q has head dimension {d}, the cache {dc}")
    max_blocks = _dims(block_table, "block_table", 2)[1]
    _have(block_table, "block_table", _I32, (B, max_blocks), dev)
    _have(seqlens_k, "seqlens_k", _I32, (B,), dev)
    max_sel = 0
    if sel is not None and n_sel is not None:
        max_sel = _dims(sel, "sel", 3)[2]
        _have(sel, "sel", _I32, (B, Hkv, max_sel), dev)
        _have(n_sel, "n_sel", _I32, (B, Hkv), dev)
    elif sel is not None or n_sel is not None:
        raise ValueError("sel and n_sel are given together or not at all")
    o = _out(o, "o", shape, _BF16, dev, stream)
    lse = _out(lse, "lse", (B, Hq, Sq), _F32, dev, stream)
    workspace = _workspace(workspace, lib.fa_decode_paged_fp8_workspace_size(B, Hq, Hkv, Sq, d),
                           dev, stream)
    st = lib.fa_decode_paged_fp8(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                 k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
                                 seqlens_k.data_ptr(), _ptr(sel), _ptr(n_sel), o.data_ptr(),
                                 lse.data_ptr(), B, Hq, Hkv, Sq, num_pages, max_blocks, max_sel,
                                 ps, d, float(scale), workspace.data_ptr(), workspace.nbytes,
                                 _stream(stream))
    _check(st, "fa_decode_paged_fp8")
    return o, lse


# ------------------------------------- between a projection and the scores --

# Sizes that depend on numbers alone are asked for once.
@functools.lru_cache(4096)
def _plan_bytes(B, Sq, Sk):
    return load_library().fa_mask_plan_size(B, Sq, Sk)


@functools.lru_cache(4096)
def _decode_scored_bytes(B, Hq, Hkv, Sk_max, d, window):
    return load_library().fa_decode_scored_workspace_size(B, Hq, Hkv, Sk_max, d, window)


def _view(t, name, shape, dev):
    """fa_heads of a bf16 tensor of that shape [B, S, H, d] with contiguous channels."""
    if not (isinstance(t, torch.Tensor) and t.dtype == _BF16 and t.get_device() == dev
            and t.shape == shape):
        _refuse(t, name, _BF16, shape, dev)
    sb, st, sh, sc = t.stride()
    if sc != 1:
        raise ValueError(f"{name} must have contiguous channels")
    return _Heads(t.data_ptr(), sb, st, sh)


def _out_view(t, name, shape, dev, stream):
    """An output [B, S, H, d] and its fa_heads: the caller's view, or a new tensor."""
    if t is not None:
        return t, _view(t, name, shape, dev)
    t = _new(shape, _BF16, dev, stream)
    _, S, H, d = shape
    return t, _Heads(t.data_ptr(), S * H * d, H * d, d)


@functools.lru_cache(None)
def _prep_bwd_bytes(d):
    return load_library().fa_qk_norm_rope_bwd_workspace_size(d)


def _rotation(positions, inv_freq, freq_axis, q_weight, k_weight, B, S, d, dev):
    """(n_axes, rot_dim) of a rotation, checked with the weights."""
    n_axes, rot = 1, 0
    if inv_freq is not None:
        half, = _dims(inv_freq, "inv_freq", 1)
        _have(inv_freq, "inv_freq", _F32, (half,), dev)
        rot = 2 * half
        if positions is not None:
            if positions.dim() == 2:
                _have(positions, "positions", _I32, (B, S), dev)
            else:
                n_axes = _dims(positions, "positions", 3)[0]
                _have(positions, "positions", _I32, (n_axes, B, S), dev)
        if freq_axis is not None:
            _have(freq_axis, "freq_axis", _U8, (half,), dev)
    elif positions is not None or freq_axis is not None:
        raise ValueError("positions and freq_axis are given with inv_freq only")
    for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _have(w, n, _BF16, (d,), dev)
    return n_axes, rot


def fa_qk_norm_rope(q, k, v=None, positions=None, inv_freq=None, freq_axis=None, q_weight=None,
                    k_weight=None, weight_offset: float = 0.0, eps: float = 1e-6,
                    interleaved: bool = False, q_out=None, k_out=None, v_out=None, row_start=None,
                    stream=None):
    """Norms of query and key heads, rotation and head-major layout in one pass (fa_qk_norm_rope).
    q [B,S,Hq,d], k and v [B,S,Hkv,d] bf16: any views with contiguous channels, for example of a
    packed projection.  q_weight/k_weight bf16 [d] (None: no norm); inv_freq fp32 [rot_dim/2] (None:
    no rotation); positions int32 [B,S] or [n_axes,B,S] (None: the rows written); freq_axis uint8
    [rot_dim/2].  k_out/v_out may be caches [B,Hkv,S_out,d] whose rows row_start[b] + s (int32 [B])
    are written.  Returns (q_out [B,Hq,S,d], k_out, v_out or None)."""
    lib, dev = load_library(), _device()
    B, S, Hq, d = _dims(q, "q", 4)
    Hkv = _dims(k, "k", 4)[2]
    vq, vk = _view(q, "q", (B, S, Hq, d), dev), _view(k, "k", (B, S, Hkv, d), dev)
    vv = None if v is None else _view(v, "v", (B, S, Hkv, d), dev)
    n_axes, rot = _rotation(positions, inv_freq, freq_axis, q_weight, k_weight, B, S, d, dev)
    rows = S
    if row_start is not None:
        _have(row_start, "row_start", _I32, (B,), dev)
        if k_out is None or (v is not None and v_out is None):
            raise ValueError("row_start is given with the caches k_out and v_out")
    if k_out is not None:
        rows = _dims(k_out, "k_out", 4)[2]
    q_out = _out(q_out, "q_out", (B, Hq, S, d), _BF16, dev, stream)
    k_out = _out(k_out, "k_out", (B, Hkv, rows, d), _BF16, dev, stream)
    if v is not None:
        v_out = _out(v_out, "v_out", (B, Hkv, rows, d), _BF16, dev, stream)
    elif v_out is not None:
        raise ValueError("v_out is given with v only")
    st = lib.fa_qk_norm_rope(vq, vk, vv, q_out.data_ptr(), k_out.data_ptr(), _ptr(v_out),
                             _ptr(row_start), rows, _ptr(q_weight), _ptr(k_weight),
                             float(weight_offset), float(eps), _ptr(positions), n_axes,
                             _ptr(inv_freq), _ptr(freq_axis), rot, int(bool(interleaved)), B, S, Hq,
                             Hkv, d, _stream(stream))
    _check(st, "fa_qk_norm_rope")
    return q_out, k_out, v_out


def fa_qk_norm_rope_bwd_workspace_size(d) -> int:
    return int(load_library().fa_qk_norm_rope_bwd_workspace_size(_int(d, "d")))


def fa_qk_norm_rope_bwd(q, k, dq_out, dk_out, dv_out=None, positions=None, inv_freq=None,
                        freq_axis=None, q_weight=None, k_weight=None, weight_offset: float = 0.0,
                        eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None, dv=None,
                        dq_weight=None, dk_weight=None, workspace=None, stream=None):
    """Gradients of fa_qk_norm_rope (without row_start): dq_out [B,Hq,S,d], dk_out/dv_out
    [B,Hkv,S,d] bf16 are those of its outputs.  dq [B,S,Hq,d], dk and dv [B,S,Hkv,d] may be views with
    contiguous channels (of a packed projection's gradient); new ones are contiguous.
    Returns (dq, dk, dv or None, dq_weight fp32 [d] or None, dk_weight or None)."""
    lib, dev = load_library(), _device()
    B, Hq, S, d = _dims(dq_out, "dq_out", 4)
    Hkv = _dims(dk_out, "dk_out", 4)[1]
    _have(dq_out, "dq_out", _BF16, (B, Hq, S, d), dev)
    _have(dk_out, "dk_out", _BF16, (B, Hkv, S, d), dev)
    n_axes, rot = _rotation(positions, inv_freq, freq_axis, q_weight, k_weight, B, S, d, dev)
    vq = None if q_weight is None else _view(q, "q", (B, S, Hq, d), dev)
    vk = None if k_weight is None else _view(k, "k", (B, S, Hkv, d), dev)
    dq, gq = _out_view(dq, "dq", (B, S, Hq, d), dev, stream)
    dk, gk = _out_view(dk, "dk", (B, S, Hkv, d), dev, stream)
    gv = None
    if dv_out is not None:
        _have(dv_out, "dv_out", _BF16, (B, Hkv, S, d), dev)
        dv, gv = _out_view(dv, "dv", (B, S, Hkv, d), dev, stream)
    elif dv is not None:
        raise ValueError("dv is given with dv_out only")
    if q_weight is not None:
        dq_weight = _out(dq_weight, "dq_weight", (d,), _F32, dev, stream)
    elif dq_weight is not None:
        raise ValueError("dq_weight is given with q_weight only")
    if k_weight is not None:
        dk_weight = _out(dk_weight, "dk_weight", (d,), _F32, dev, stream)
    elif dk_weight is not None:
        raise ValueError("dk_weight is given with k_weight only")
    nbytes = 0
    if q_weight is not None or k_weight is not None:
        workspace = _workspace(workspace, _prep_bwd_bytes(d), dev, stream)
        nbytes = workspace.nbytes
    st = lib.fa_qk_norm_rope_bwd(vq, vk, dq_out.data_ptr(), dk_out.data_ptr(), _ptr(dv_out), gq, gk,
                                 gv, _ptr(dq_weight), _ptr(dk_weight), _ptr(q_weight),
                                 _ptr(k_weight), float(weight_offset), float(eps), _ptr(positions),
                                 n_axes, _ptr(inv_freq), _ptr(freq_axis), rot,
                                 int(bool(interleaved)), B, S, Hq, Hkv, d, _ptr(workspace), nbytes,
                                 _stream(stream))
    _check(st, "fa_qk_norm_rope_bwd")
    return dq, dk, dv, dq_weight, dk_weight


# ------------------------------------------------ capped and biased scores --

def fa_row_bounds(B: int, Sq: int, Sk: int, causal: bool, window: int = 0, cu_docs=None, prefix=None,
                  row_lo=None, row_hi=None, stream=None):
    """Visible keys [lo, hi) of every row under documents, prefixes and a window (fa_row_bounds).
    cu_docs int32 [n_docs+1] offsets into the B * Sk flattened positions; prefix int32 [n_docs] ([B]
    without cu_docs), negative for padding.  Returns (row_lo, row_hi) int32 [B,Sq]."""
    lib, dev = load_library(), _device()
    B, Sq, Sk = _int(B, "B"), _int(Sq, "Sq"), _int(Sk, "Sk")
    if min(B, Sq, Sk) < 1:
        raise ValueError(f"sizes must be >= 1 (B={B} Sq={Sq} Sk={Sk})")
    n_docs = 0
    if cu_docs is not None:
        n_docs = _dims(cu_docs, "cu_docs", 1)[0] - 1
        _have(cu_docs, "cu_docs", _I32, (n_docs + 1,), dev)
    if prefix is not None:
        _have(prefix, "prefix", _I32, (B if cu_docs is None else n_docs,), dev)
    row_lo = _out(row_lo, "row_lo", (B, Sq), _I32, dev, stream)
    row_hi = _out(row_hi, "row_hi", (B, Sq), _I32, dev, stream)
    st = lib.fa_row_bounds(_ptr(cu_docs), _ptr(prefix), n_docs, row_lo.data_ptr(), row_hi.data_ptr(),
                           B, Sq, Sk, int(bool(causal)), _int(window, "window"), _stream(stream))
    _check(st, "fa_row_bounds")
    return row_lo, row_hi


def fa_mask_plan_size(B, Sq, Sk) -> int:
    return int(load_library().fa_mask_plan_size(_int(B, "B"), _int(Sq, "Sq"), _int(Sk, "Sk")))


def fa_mask_plan(row_lo, row_hi, Sk: int, plan=None, stream=None):
    """The tile plan of row intervals (fa_mask_plan): row_lo, row_hi int32 [B,Sq].  Returns the plan,
    a uint8 tensor of fa_mask_plan_size(B, Sq, Sk) bytes for fa_fwd_scored and fa_bwd_scored of these sizes."""
    lib, dev = load_library(), _device()
    B, Sq = _dims(row_lo, "row_lo", 2)
    Sk = _int(Sk, "Sk")
    _have(row_lo, "row_lo", _I32, (B, Sq), dev)
    _have(row_hi, "row_hi", _I32, (B, Sq), dev)
    nbytes = _plan_bytes(B, Sq, Sk)
    plan = _out(plan, "plan", (nbytes,), _U8, dev, stream)
    st = lib.fa_mask_plan(row_lo.data_ptr(), row_hi.data_ptr(), B, Sq, Sk, plan.data_ptr(), nbytes,
                          _stream(stream))
    _check(st, "fa_mask_plan")
    plan.fa_sizes = B, Sq, Sk  # for the calls that take it: other sizes may have as many bytes
    return plan


def _scored_args(q, k, v, slopes, plan, dev):
    """(B, Hq, Hkv, Sq, Sk, d, plan bytes) of an attention call on capped or biased scores."""
    B, Hq, Sq, d = _dims(q, "q", 4)
    _, Hkv, Sk, _ = _dims(k, "k", 4)
    _have(q, "q", _BF16, (B, Hq, Sq, d), dev)
    _have(k, "k", _BF16, (B, Hkv, Sk, d), dev)
    _have(v, "v", _BF16, (B, Hkv, Sk, d), dev)
    if slopes is not None:
        _have(slopes, "slopes", _F32, (Hq,), dev)
    if plan is None:
        return B, Hq, Hkv, Sq, Sk, d, 0
    nbytes = _plan_bytes(B, Sq, Sk)
    _have(plan, "plan", _U8, (nbytes,), dev)
    if getattr(plan, "fa_sizes", (B, Sq, Sk)) != (B, Sq, Sk):
        raise ValueError(f"plan was made for B, Sq, Sk = {plan.fa_sizes}, the call has {(B, Sq, Sk)}")
    return B, Hq, Hkv, Sq, Sk, d, nbytes


@functools.lru_cache(4096)
def _fwd_scored_bytes(B, Hq, Hkv, Sq, Sk, d):
    return load_library().fa_fwd_scored_workspace_size(B, Hq, Hkv, Sq, Sk, d)


def fa_fwd_scored_workspace_size(B, Hq, Hkv, Sq, Sk, d) -> int:
    return int(load_library().fa_fwd_scored_workspace_size(
        _int(B, "B"), _int(Hq, "Hq"), _int(Hkv, "Hkv"), _int(Sq, "Sq"), _int(Sk, "Sk"), _int(d, "d")))


def fa_fwd_scored(q, k, v, causal: bool, scale: float, softcap: float = 0.0, slopes=None, plan=None,
                  o=None, lse=None, workspace=None, stream=None):
    """Attention on capped and biased scores (fa_fwd_scored): q [B,Hq,Sq,d], k/v [B,Hkv,Sk,d] bf16;
    softcap 0 for none; slopes fp32 [Hq] of the bias -slope * distance; plan from fa_mask_plan.  The
    workspace is fa_fwd_scored_workspace_size(B, Hq, Hkv, Sq, Sk, d) bytes.  Returns (o, lse)."""
    lib, dev = load_library(), _device()
    B, Hq, Hkv, Sq, Sk, d, nplan = _scored_args(q, k, v, slopes, plan, dev)
    o = _out(o, "o", (B, Hq, Sq, d), _BF16, dev, stream)
    lse = _out(lse, "lse", (B, Hq, Sq), _F32, dev, stream)
    nbytes = _fwd_scored_bytes(B, Hq, Hkv, Sq, Sk, d)
    if nbytes or workspace is not None:
        workspace = _workspace(workspace, nbytes, dev, stream)
        nbytes = workspace.nbytes
    st = lib.fa_fwd_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B,
                           Hq, Hkv, Sq, Sk, d, int(bool(causal)), float(scale), float(softcap),
                           _ptr(slopes), _ptr(plan), nplan, _ptr(workspace), nbytes, _stream(stream))
    _check(st, "fa_fwd_scored")
    return o, lse


@functools.lru_cache(4096)
def _bwd_scored_bytes(B, Hq, Hkv, Sq, Sk, d):
    return load_library().fa_bwd_scored_workspace_size(B, Hq, Hkv, Sq, Sk, d)


def fa_bwd_scored_workspace_size(B, Hq, Hkv, Sq, Sk, d) -> int:
    return int(load_library().fa_bwd_scored_workspace_size(
        _int(B, "B"), _int(Hq, "Hq"), _int(Hkv, "Hkv"), _int(Sq, "Sq"), _int(Sk, "Sk"), _int(d, "d")))


def fa_bwd_scored(q, k, v, o, dout, lse, causal: bool, scale: float, softcap: float = 0.0,
                  slopes=None, plan=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """dQ, dK, dV of fa_fwd_scored (fa_bwd_scored), with the forward's arguments.  The workspace is
    fa_bwd_scored_workspace_size(B, Hq, Hkv, Sq, Sk, d) bytes; fa_bwd_workspace_size(B, Hq, Sq, d) are
    enough, but few keys are then not split over the GPU.  Returns (dq, dk, dv)."""
    lib, dev = load_library(), _device()
    B, Hq, Hkv, Sq, Sk, d, nplan = _scored_args(q, k, v, slopes, plan, dev)
    _have(o, "o", _BF16, (B, Hq, Sq, d), dev)
    _have(dout, "dout", _BF16, (B, Hq, Sq, d), dev)
    _have(lse, "lse", _F32, (B, Hq, Sq), dev)
    dq = _out(dq, "dq", (B, Hq, Sq, d), _BF16, dev, stream)
    dk = _out(dk, "dk", (B, Hkv, Sk, d), _BF16, dev, stream)
    dv = _out(dv, "dv", (B, Hkv, Sk, d), _BF16, dev, stream)
    workspace = _workspace(workspace, _bwd_scored_bytes(B, Hq, Hkv, Sq, Sk, d), dev, stream)
    st = lib.fa_bwd_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                           lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv,
                           Sq, Sk, d, int(bool(causal)), float(scale), float(softcap), _ptr(slopes),
                           _ptr(plan), nplan, workspace.data_ptr(), workspace.nbytes,
                           _stream(stream))
    _check(st, "fa_bwd_scored")
    return dq, dk, dv


def fa_decode_scored_workspace_size(B, Hq, Hkv, Sk_max, d, window=0) -> int:
    return int(load_library().fa_decode_scored_workspace_size(
        _int(B, "B"), _int(Hq, "Hq"), _int(Hkv, "Hkv"), _int(Sk_max, "Sk_max"), _int(d, "d"),
        _int(window, "window")))


def fa_decode_scored(q, k_cache, v_cache, seqlens_k, scale: float, softcap: float = 0.0, slopes=None,
                     window: int = 0, k_start=None, o=None, lse=None, workspace=None, stream=None):
    """Single-query decode on capped and biased scores (fa_decode_scored): q [B,Hq,1,d],
    k_cache/v_cache [B,Hkv,Sk_max,d] bf16, seqlens_k int32 [B]; window: how many last keys are seen
    (0: all); k_start int32 [B]: first key.  Returns (o [B,Hq,1,d], lse [B,Hq])."""
    lib, dev = load_library(), _device()
    B, Hq, one, d = _dims(q, "q", 4)
    _, Hkv, Sk_max, _ = _dims(k_cache, "k_cache", 4)
    if one != 1:
        raise ValueError(f"q must be [B, Hq, 1, d], got {tuple(q.shape)}")
    _have(q, "q", _BF16, (B, Hq, 1, d), dev)
    _have(k_cache, "k_cache", _BF16, (B, Hkv, Sk_max, d), dev)
    _have(v_cache, "v_cache", _BF16, (B, Hkv, Sk_max, d), dev)
    _have(seqlens_k, "seqlens_k", _I32, (B,), dev)
    if k_start is not None:
        _have(k_start, "k_start", _I32, (B,), dev)
    if slopes is not None:
        _have(slopes, "slopes", _F32, (Hq,), dev)
    window = _int(window, "window")
    o = _out(o, "o", (B, Hq, 1, d), _BF16, dev, stream)
    lse = _out(lse, "lse", (B, Hq), _F32, dev, stream)
    nbytes = _decode_scored_bytes(B, Hq, Hkv, Sk_max, d, window)
    if nbytes or workspace is not None:
        workspace = _workspace(workspace, nbytes, dev, stream)
        nbytes = workspace.nbytes
    st = lib.fa_decode_scored(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), o.data_ptr(),
                              lse.data_ptr(), seqlens_k.data_ptr(), _ptr(k_start), B, Hq, Hkv,
                              Sk_max, d, float(scale), float(softcap), _ptr(slopes), window,
                              _ptr(workspace), nbytes, _stream(stream))
    _check(st, "fa_decode_scored")
    return o, lse


def fa_device_status(clear: bool = True):
    """(status, raw word) of the device status words; synchronises the device."""
    lib = load_library()
    w = ctypes.c_uint(0)
    st = lib.fa_device_status(ctypes.byref(w), int(bool(clear)))
    return st, w.value


def fa_selftest_wait_timeout(stream=None):
    """Run the bounded-wait self-test (about 1 s): returns the two flags the
    kernel sets (1 = that wait reported failure).  fa_device_status() then
    reports the recorded timeout."""
    lib = load_library()
    res = torch.zeros(4, dtype=torch.int32, device="cuda")
    _check(lib.fa_selftest_wait_timeout(_ptr(res), _stream(stream)), "fa_selftest_wait_timeout")
    return [int(x) for x in res[:2].cpu()]


def fa_profile_next_launch(start=None, stop=None):
    """Arm the one-shot hook: the next fa_* call on this thread records the two
    torch.cuda.Event objects around its main kernel (None, None disarms)."""
    lib = load_library()
    a = None if start is None else ctypes.c_void_p(start.cuda_event)
    b = None if stop is None else ctypes.c_void_p(stop.cuda_event)
    _check(lib.fa_profile_next_launch(a, b), "fa_profile_next_launch")


def version() -> str:
    return load_library().fa_version().decode()
