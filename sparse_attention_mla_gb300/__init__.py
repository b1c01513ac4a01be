"""GB300-native (sm_103a) DeepSeek Sparse Attention hot path.

Thin Python binding over the C ABI of ``libdsa.so`` (see ``include/dsa.h``).
The functions carry the C entry points' names and only marshal arguments:
torch supplies device memory and the current CUDA stream; every step of the
computation runs in the library's CUDA kernels.  There is no CPU fallback: if
the library is missing or the device is not sm_103, the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import re
import threading

import torch

from .build_ext import LIB as _LIB_PATH
from .build_ext import INCLUDE as _INCLUDE

__all__ = [
    "DsaError",
    "load_library",
    "declared_symbols",
    "dsa_packed_metadata",
    "dsa_packed_metadata_cp",
    "dsa_indexer_topk",
    "dsa_indexer_topk_cp",
    "dsa_indexer_topk_with_scores",
    "dsa_indexer_topk_scored",
    "dsa_indexer_kl",
    "dsa_kpool_metadata",
    "dsa_kpool_pool",
    "dsa_kpool_topk",
    "dsa_kpool_unpool_grad",
    "dsa_sparse_mla_fwd",
    "dsa_sparse_mla_bwd",
    "dsa_sparse_mla_bwd_noalloc",
    "dsa_sparse_mla_bwd_noalloc_read_status",
    "dsa_paged_slots",
    "dsa_norm_rope_fwd",
    "dsa_norm_rope_bwd",
    "dsa_rope_frequencies",
    "dsa_paged_mla",
    "dsa_paged_indexer_topk",
    "dsa_paged_quantize",
    "dsa_paged_dequantize",
    "dsa_paged_mla_quant",
    "dsa_read_device_status",
    "dsa_set_wait_limit_cycles",
    "workspace_size",
    "paged_workspace_size",
    "paged_quant_row_bytes",
]

DSA_OK = 0
STATUS_NAMES = {
    0: "DSA_OK",
    1: "DSA_ERR_UNSUPPORTED",
    2: "DSA_ERR_DTYPE",
    3: "DSA_ERR_INVALID_ARGUMENT",
    4: "DSA_ERR_WORKSPACE",
    5: "DSA_ERR_CUDA",
    6: "DSA_ERR_DEVICE_INDEX",
    7: "DSA_ERR_TIMEOUT",
    8: "DSA_ERR_CAPACITY",
}


class DsaError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {message}")


_lib = None
_lock = threading.Lock()
_P = ctypes.c_void_p
_I = ctypes.c_int32
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_D = ctypes.c_double
_L = ctypes.c_int64


def declared_symbols() -> list[str]:
    """Function names declared in include/*.h (the ABI surface)."""
    names = []
    for fn in sorted(os.listdir(_INCLUDE)):
        if fn.endswith(".h"):
            text = open(os.path.join(_INCLUDE, fn)).read()
            names += re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*(dsa_[a-z0-9_]+)\s*\(", text, re.M)
    return sorted(set(names))


def load_library(path: str | None = None):
    """Load libdsa.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or _LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} not found: build the CUDA library first "
                "(python -m sparse_attention_mla_gb300.build_ext, or __graft_entry__.build())")
        lib = ctypes.CDLL(path)
        lib.dsa_status_string.restype = ctypes.c_char_p
        lib.dsa_status_string.argtypes = [ctypes.c_int]
        lib.dsa_last_error_message.restype = ctypes.c_char_p
        lib.dsa_last_error_message.argtypes = []
        lib.dsa_abi_version.restype = _I
        lib.dsa_packed_metadata.argtypes = [_P, _I, _I, _P, _P, _P, _P, _P]
        lib.dsa_packed_metadata_cp.argtypes = [_P, _P, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P]
        lib.dsa_indexer_topk_workspace_size.argtypes = [_I, _I]
        lib.dsa_indexer_topk_workspace_size.restype = _SZ
        lib.dsa_indexer_topk.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]
        lib.dsa_indexer_topk_cp.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]
        lib.dsa_indexer_topk_scored.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]
        lib.dsa_indexer_topk_with_scores.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _I, _I, _P,
                                                     _SZ, _P]
        lib.dsa_sparse_mla_fwd_workspace_size.argtypes = [_I, _I]
        lib.dsa_sparse_mla_fwd_workspace_size.restype = _SZ
        lib.dsa_sparse_mla_fwd.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P, _SZ, _P]
        lib.dsa_sparse_mla_bwd_workspace_size.argtypes = [_I, _I, _I]
        lib.dsa_sparse_mla_bwd_workspace_size.restype = _SZ
        lib.dsa_sparse_mla_bwd.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P, _P, _P,
                                           _P, _P, _I, _P, _P, _SZ, _P]
        lib.dsa_read_device_status.argtypes = [_P, _P, _P]
        lib.dsa_indexer_kl_workspace_size.argtypes = [_I, _I]
        lib.dsa_indexer_kl_workspace_size.restype = _SZ
        lib.dsa_indexer_kl.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _I, _P,
                                       _SZ, _P]
        lib.dsa_indexer_kl.restype = ctypes.c_int
        lib.dsa_set_wait_limit_cycles.argtypes = [ctypes.c_int64]
        lib.dsa_set_wait_limit_cycles.restype = ctypes.c_int64
        lib.dsa_sparse_mla_bwd_noalloc_max_topk.restype = _I
        lib.dsa_sparse_mla_bwd_noalloc_max_topk.argtypes = []
        lib.dsa_sparse_mla_bwd_noalloc.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P,
                                                   _P, _P, _P, _P, _I, _P, _P]
        lib.dsa_sparse_mla_bwd_noalloc.restype = ctypes.c_int
        lib.dsa_sparse_mla_bwd_noalloc_read_status.argtypes = [_P, _P]
        lib.dsa_sparse_mla_bwd_noalloc_read_status.restype = ctypes.c_int
        lib.dsa_kpool_metadata.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P]
        lib.dsa_kpool_pool.argtypes = [_P, _I, _I, _P, _P, _I, _I, _I, _P, _P]
        lib.dsa_kpool_topk_workspace_size.argtypes = [_I, _I]
        lib.dsa_kpool_topk_workspace_size.restype = _SZ
        lib.dsa_kpool_topk.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]
        lib.dsa_kpool_unpool_grad.argtypes = [_P, _I, _I, _P, _P, _I, _I, _I, _P, _P]
        for name in ("dsa_kpool_metadata", "dsa_kpool_pool", "dsa_kpool_topk", "dsa_kpool_unpool_grad"):
            getattr(lib, name).restype = ctypes.c_int
        for name in ("dsa_packed_metadata", "dsa_indexer_topk", "dsa_indexer_topk_with_scores", "dsa_indexer_topk_scored",
                     "dsa_indexer_topk_cp",
                     "dsa_sparse_mla_fwd", "dsa_sparse_mla_bwd", "dsa_read_device_status"):
            getattr(lib, name).restype = ctypes.c_int
        lib.dsa_paged_slots.argtypes = [_P, _P, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        lib.dsa_norm_rope_fwd.argtypes = [_P, _L, _L, _I, _I, _I, _I, _I, _P, _P, _F, _I, _I, _I, _P, _P, _F, _P, _L,
                                          _L, _P, _L, _P, _SZ, _P]
        lib.dsa_norm_rope_bwd_workspace_size.argtypes = [_I]
        lib.dsa_norm_rope_bwd_workspace_size.restype = _SZ
        lib.dsa_norm_rope_bwd.argtypes = [_P, _L, _L, _P, _L, _L, _I, _I, _I, _I, _I, _P, _F, _I, _I, _I, _P, _P, _F,
                                          _P, _L, _L, _P, _P, _I, _P, _SZ, _P]
        lib.dsa_rope_frequencies.argtypes = [_I, _D, _D, _I, _D, _D, _P, _P]
        lib.dsa_paged_mla_workspace_size.argtypes = []
        lib.dsa_paged_mla_workspace_size.restype = _SZ
        lib.dsa_paged_mla.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P,
                                      _SZ, _P]
        lib.dsa_paged_indexer_topk_workspace_size.argtypes = [_I, _I]
        lib.dsa_paged_indexer_topk_workspace_size.restype = _SZ
        lib.dsa_paged_indexer_topk.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P,
                                               _SZ, _P]
        lib.dsa_paged_quant_row_bytes.argtypes = [_I, _I, _I]
        lib.dsa_paged_quant_row_bytes.restype = _SZ
        lib.dsa_paged_quantize.argtypes = [_P, _L, _I, _I, _I, _I, _P, _L, _P, _P, _SZ, _P]
        lib.dsa_paged_dequantize.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _L, _P, _SZ, _P]
        lib.dsa_paged_mla_quant_workspace_size.argtypes = []
        lib.dsa_paged_mla_quant_workspace_size.restype = _SZ
        lib.dsa_paged_mla_quant.argtypes = [_P] * 7 + [_I] * 10 + [_F, _P, _P, _P, _P, _SZ, _P]
        for name in ("dsa_paged_slots", "dsa_norm_rope_fwd", "dsa_norm_rope_bwd", "dsa_rope_frequencies",
                     "dsa_paged_mla", "dsa_paged_indexer_topk", "dsa_paged_quantize", "dsa_paged_dequantize",
                     "dsa_paged_mla_quant"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def _check(status: int, where: str):
    if status != DSA_OK:
        lib = load_library()
        raise DsaError(status, where, lib.dsa_last_error_message().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, dtype, ndim=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def workspace_size(kind: str, T: int, H_or_K: int, K: int | None = None) -> int:
    """Workspace bytes: ("fwd", T, H), ("indexer", T, K) or ("bwd", T, H, K)."""
    lib = load_library()
    if kind == "bwd":
        if K is None:
            raise ValueError('workspace_size("bwd", T, H, K) needs the top-k width K')
        return int(lib.dsa_sparse_mla_bwd_workspace_size(int(T), int(H_or_K), int(K)))
    fn = {"fwd": lib.dsa_sparse_mla_fwd_workspace_size, "indexer": lib.dsa_indexer_topk_workspace_size}[kind]
    return int(fn(int(T), int(H_or_K)))


def _workspace(kind, T, x, device, workspace, K=None):
    need = workspace_size(kind, T, x, K)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    return workspace, workspace.numel()


def dsa_packed_metadata(cu_seqlens: torch.Tensor, total_tokens: int):
    """cu_seqlens int32 [nseq+1] (CUDA) -> (seq_start [T], causal_len [T], max_seqlen, all_rows_nonempty)."""
    lib = load_library()
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    dev = cu_seqlens.device
    T = int(total_tokens)
    start = torch.empty(T, dtype=torch.int32, device=dev)
    clen = torch.empty(T, dtype=torch.int32, device=dev)
    mx = ctypes.c_int32(0)
    ne = ctypes.c_int32(0)
    _check(lib.dsa_packed_metadata(_ptr(cu_seqlens), cu_seqlens.numel() - 1, T, _ptr(start), _ptr(clen),
                                   ctypes.byref(mx), ctypes.byref(ne), _stream(dev)), "dsa_packed_metadata")
    return start, clen, mx.value, ne.value


def dsa_packed_metadata_cp(cu_seqlens: torch.Tensor, total_key_tokens: int, query_indices=None,
                           cu_seqlens_padded=None, padding_mask=None, T_q: int | None = None):
    """Context-parallel metadata: rank-local query rows (global padded coordinates `query_indices`,
    identity when None) against gathered global keys -> (seq_start [T_q], causal_len [T_q],
    max_seqlen, all_rows_nonempty).  padding_mask: bool/uint8 [T_q], True marks a padding row."""
    lib = load_library()
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    dev = cu_seqlens.device
    if cu_seqlens_padded is not None:
        _need(cu_seqlens_padded, "cu_seqlens_padded", torch.int32, 1, dev)
        if cu_seqlens_padded.numel() != cu_seqlens.numel():
            raise ValueError("cu_seqlens_padded must have as many entries as cu_seqlens")
    if query_indices is not None:
        _need(query_indices, "query_indices", torch.int32, 1, dev)
    if T_q is None:
        T_q = query_indices.numel() if query_indices is not None else int(total_key_tokens)
    T_q = int(T_q)
    if query_indices is not None and query_indices.numel() != T_q:
        raise ValueError("query_indices must have T_q entries")
    if padding_mask is not None:
        if padding_mask.dtype == torch.bool:
            padding_mask = padding_mask.view(torch.uint8)
        _need(padding_mask, "padding_mask", torch.uint8, 1, dev)
        if padding_mask.numel() != T_q:
            raise ValueError("padding_mask must have T_q entries")
    start = torch.empty(T_q, dtype=torch.int32, device=dev)
    clen = torch.empty(T_q, dtype=torch.int32, device=dev)
    mx = ctypes.c_int32(0)
    ne = ctypes.c_int32(0)
    _check(lib.dsa_packed_metadata_cp(_ptr(cu_seqlens), _ptr(cu_seqlens_padded), cu_seqlens.numel() - 1,
                                      int(total_key_tokens), _ptr(query_indices), _ptr(padding_mask), T_q, _ptr(start),
                                      _ptr(clen), ctypes.byref(mx), ctypes.byref(ne), _stream(dev)),
           "dsa_packed_metadata_cp")
    return start, clen, mx.value, ne.value


def dsa_indexer_topk_cp(q_idx, k_idx, head_weights, seq_start, causal_len, K: int, topk_idx=None, topk_len=None,
                        workspace=None):
    """Indexer top-k for rank-local rows against gathered global keys: row r's window is
    [seq_start[r], seq_start[r] + causal_len[r] - 1] -> (topk_idx int32 [T_q, K], topk_len int32 [T_q])."""
    lib = load_library()
    _need(q_idx, "q_idx", torch.bfloat16, 3)
    dev = q_idx.device
    _need(k_idx, "k_idx", torch.bfloat16, 2, dev)
    _need(head_weights, "head_weights", torch.float32, 2, dev)
    _need(seq_start, "seq_start", torch.int32, 1, dev)
    _need(causal_len, "causal_len", torch.int32, 1, dev)
    T, Hi, Di = q_idx.shape
    Tk = k_idx.shape[0]
    if topk_idx is None:
        topk_idx = torch.empty(T, K, dtype=torch.int32, device=dev)
    if topk_len is None:
        topk_len = torch.empty(T, dtype=torch.int32, device=dev)
    ws, wsb = _workspace("indexer", T, K, dev, workspace)
    _check(lib.dsa_indexer_topk_cp(_ptr(q_idx), _ptr(k_idx), _ptr(head_weights), _ptr(seq_start), _ptr(causal_len),
                                   T, Tk, Hi, Di, int(K), _ptr(topk_idx), _ptr(topk_len), _ptr(ws), wsb,
                                   _stream(dev)),
           "dsa_indexer_topk_cp")
    return topk_idx, topk_len


def dsa_indexer_topk(q_idx, k_idx, head_weights, seq_start, K: int, topk_idx=None, topk_len=None,
                     workspace=None, with_len: bool = True):
    """Fused indexer score + causal top-k -> (topk_idx int32 [T,K], topk_len int32 [T] or None)."""
    lib = load_library()
    _need(q_idx, "q_idx", torch.bfloat16, 3)
    dev = q_idx.device
    _need(k_idx, "k_idx", torch.bfloat16, 2, dev)
    _need(head_weights, "head_weights", torch.float32, 2, dev)
    _need(seq_start, "seq_start", torch.int32, 1, dev)
    T, Hi, Di = q_idx.shape
    Tk = k_idx.shape[0]
    if topk_idx is None:
        topk_idx = torch.empty(T, K, dtype=torch.int32, device=dev)
    if topk_len is None and with_len:
        topk_len = torch.empty(T, dtype=torch.int32, device=dev)
    ws, wsb = _workspace("indexer", T, K, dev, workspace)
    _check(lib.dsa_indexer_topk(_ptr(q_idx), _ptr(k_idx), _ptr(head_weights), _ptr(seq_start), T, Tk, Hi, Di,
                                int(K), _ptr(topk_idx), _ptr(topk_len), _ptr(ws), wsb, _stream(dev)),
           "dsa_indexer_topk")
    return topk_idx, topk_len


def dsa_indexer_topk_scored(q_idx, k_idx, head_weights, seq_start, K: int, causal_len=None, topk_idx=None,
                            topk_len=None, topk_score=None, workspace=None):
    """dsa_indexer_topk (causal_len None) or dsa_indexer_topk_cp that also returns each selected slot's fp32
    score -> (topk_idx int32 [T,K], topk_len int32 [T], topk_score fp32 [T,K], -inf after the prefix)."""
    lib = load_library()
    _need(q_idx, "q_idx", torch.bfloat16, 3)
    dev = q_idx.device
    _need(k_idx, "k_idx", torch.bfloat16, 2, dev)
    _need(head_weights, "head_weights", torch.float32, 2, dev)
    _need(seq_start, "seq_start", torch.int32, 1, dev)
    if causal_len is not None:
        _need(causal_len, "causal_len", torch.int32, 1, dev)
    T, Hi, Di = q_idx.shape
    Tk = k_idx.shape[0]
    if topk_idx is None:
        topk_idx = torch.empty(T, K, dtype=torch.int32, device=dev)
    if topk_len is None:
        topk_len = torch.empty(T, dtype=torch.int32, device=dev)
    if topk_score is None:
        topk_score = torch.empty(T, K, dtype=torch.float32, device=dev)
    _need(topk_score, "topk_score", torch.float32, 2, dev)
    ws, wsb = _workspace("indexer", T, K, dev, workspace)
    _check(lib.dsa_indexer_topk_scored(_ptr(q_idx), _ptr(k_idx), _ptr(head_weights), _ptr(seq_start),
                                       _ptr(causal_len), T, Tk, Hi, Di, int(K), _ptr(topk_idx), _ptr(topk_len),
                                       _ptr(topk_score), _ptr(ws), wsb, _stream(dev)),
           "dsa_indexer_topk_scored")
    return topk_idx, topk_len, topk_score


def dsa_indexer_topk_with_scores(q_idx, k_idx, head_weights, seq_start, K: int, score_row0: int,
                                 score_rows: int, workspace=None):
    """Diagnostic form of dsa_indexer_topk -> (topk_idx, topk_len, scores fp32 [score_rows, T_k]): the
    fp32 score of every window key of rows score_row0 .. score_row0 + score_rows - 1 (NaN elsewhere)."""
    lib = load_library()
    _need(q_idx, "q_idx", torch.bfloat16, 3)
    dev = q_idx.device
    _need(k_idx, "k_idx", torch.bfloat16, 2, dev)
    _need(head_weights, "head_weights", torch.float32, 2, dev)
    _need(seq_start, "seq_start", torch.int32, 1, dev)
    T, Hi, Di = q_idx.shape
    Tk = k_idx.shape[0]
    topk_idx = torch.empty(T, K, dtype=torch.int32, device=dev)
    topk_len = torch.empty(T, dtype=torch.int32, device=dev)
    scores = torch.full((score_rows, Tk), float("nan"), dtype=torch.float32, device=dev)
    ws, wsb = _workspace("indexer", T, K, dev, workspace)
    _check(lib.dsa_indexer_topk_with_scores(_ptr(q_idx), _ptr(k_idx), _ptr(head_weights), _ptr(seq_start), T, Tk,
                                            Hi, Di, int(K), _ptr(topk_idx), _ptr(topk_len), _ptr(scores),
                                            int(score_row0), int(score_rows), _ptr(ws), wsb, _stream(dev)),
           "dsa_indexer_topk_with_scores")
    return topk_idx, topk_len, scores


def dsa_indexer_kl(q_idx, k_idx, head_weights, topk_idx, attn_prob, coeff: float, topk_len=None, kl=None,
                   dq_idx=None, dw=None, dk_idx_accum=None, accumulate: bool = False, workspace=None,
                   topk_score=None):
    """Indexer KL auxiliary loss over each row's selected slots and its gradient -> (kl fp32 [T],
    dq_idx bf16 [T,Hi,Di], dw fp32 [T,Hi], dk_idx_accum fp32 [T_k,Di]); the gradients are those of
    coeff * sum_t kl[t].  attn_prob: fp32 [T, K], e.g. from dsa_sparse_mla_bwd(attn_prob=True).
    topk_score: fp32 [T, K] or None, the slots' indexer scores (dsa_indexer_topk_scored), read instead
    of formed again."""
    lib = load_library()
    _need(q_idx, "q_idx", torch.bfloat16, 3)
    dev = q_idx.device
    _need(k_idx, "k_idx", torch.bfloat16, 2, dev)
    _need(head_weights, "head_weights", torch.float32, 2, dev)
    _need(topk_idx, "topk_idx", torch.int32, 2, dev)
    _need(attn_prob, "attn_prob", torch.float32, 2, dev)
    if topk_len is not None:
        _need(topk_len, "topk_len", torch.int32, 1, dev)
    T, Hi, Di = q_idx.shape
    Tk = k_idx.shape[0]
    K = topk_idx.shape[1]
    if attn_prob.shape != topk_idx.shape:
        raise ValueError("attn_prob must have the shape of topk_idx")
    if topk_score is not None:
        _need(topk_score, "topk_score", torch.float32, 2, dev)
        if topk_score.shape != topk_idx.shape:
            raise ValueError("topk_score must have the shape of topk_idx")
    kl = torch.empty(T, dtype=torch.float32, device=dev) if kl is None else kl
    dq_idx = torch.empty(T, Hi, Di, dtype=torch.bfloat16, device=dev) if dq_idx is None else dq_idx
    dw = torch.empty(T, Hi, dtype=torch.float32, device=dev) if dw is None else dw
    if dk_idx_accum is None:
        if accumulate:
            raise ValueError("accumulate=True needs an existing dk_idx_accum")
        dk_idx_accum = torch.empty(Tk, Di, dtype=torch.float32, device=dev)
    for t_, n_, dt_ in ((kl, "kl", torch.float32), (dq_idx, "dq_idx", torch.bfloat16), (dw, "dw", torch.float32),
                        (dk_idx_accum, "dk_idx_accum", torch.float32)):
        _need(t_, n_, dt_, None, dev)
    if workspace is None:
        workspace = torch.empty(max(int(lib.dsa_indexer_kl_workspace_size(T, K)), 256), dtype=torch.uint8,
                                device=dev)
    _check(lib.dsa_indexer_kl(_ptr(q_idx), _ptr(k_idx), _ptr(head_weights), _ptr(topk_idx), _ptr(topk_len),
                              _ptr(attn_prob), _ptr(topk_score), T, Tk, Hi, Di, K, float(coeff), _ptr(kl), _ptr(dq_idx), _ptr(dw),
                              _ptr(dk_idx_accum), 1 if accumulate else 0, _ptr(workspace), workspace.numel(),
                              _stream(dev)),
           "dsa_indexer_kl")
    return kl, dq_idx, dw, dk_idx_accum


class KPoolMeta:
    """Pool coordinates of a packed batch (dsa_kpool_metadata): pool size, per-sequence pool
    offsets (device int32 [nseq+1]), per-token pool_start / n_pools / tail_start (device int32 [T])
    and the total number of pools."""

    def __init__(self, cu_seqlens, pool, pool_cu, pool_start, n_pools, tail_start, total_pools):
        self.cu_seqlens, self.pool, self.pool_cu = cu_seqlens, pool, pool_cu
        self.pool_start, self.n_pools, self.tail_start, self.total_pools = pool_start, n_pools, tail_start, total_pools

    @property
    def num_seqs(self) -> int:
        return self.cu_seqlens.numel() - 1

    @property
    def total_tokens(self) -> int:
        return self.pool_start.numel()


def dsa_kpool_metadata(cu_seqlens: torch.Tensor, total_tokens: int, pool: int = 4) -> KPoolMeta:
    """k-pool coordinates: pools of `pool` consecutive tokens of each packed sequence (GLM-5.3-Flash)."""
    lib = load_library()
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    dev = cu_seqlens.device
    T = int(total_tokens)
    pool_cu = torch.empty(cu_seqlens.numel(), dtype=torch.int32, device=dev)
    ps = torch.empty(T, dtype=torch.int32, device=dev)
    npl = torch.empty(T, dtype=torch.int32, device=dev)
    ts = torch.empty(T, dtype=torch.int32, device=dev)
    total = ctypes.c_int32(0)
    _check(lib.dsa_kpool_metadata(_ptr(cu_seqlens), cu_seqlens.numel() - 1, T, int(pool), _ptr(pool_cu), _ptr(ps),
                                  _ptr(npl), _ptr(ts), ctypes.byref(total), _stream(dev)), "dsa_kpool_metadata")
    return KPoolMeta(cu_seqlens, int(pool), pool_cu, ps, npl, ts, total.value)


def dsa_kpool_pool(x: torch.Tensor, meta: KPoolMeta, out=None):
    """Pooled rows of x (bf16 [T, D]) -> bf16 [total_pools, D]: the mean of each pool's token rows."""
    lib = load_library()
    _need(x, "x", torch.bfloat16, 2)
    dev = x.device
    T, D = x.shape
    if out is None:
        out = torch.empty(meta.total_pools, D, dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, 2, dev)
    _check(lib.dsa_kpool_pool(_ptr(x), T, D, _ptr(meta.cu_seqlens), _ptr(meta.pool_cu), meta.num_seqs, meta.pool,
                              meta.total_pools, _ptr(out), _stream(dev)), "dsa_kpool_pool")
    return out


def dsa_kpool_topk(q_idx, k_pool, head_weights, meta: KPoolMeta, K: int = 2048, topk_idx=None, topk_len=None,
                   workspace=None):
    """k-pool selection -> (topk_idx int32 [T, K + pool - 1], topk_len int32 [T]): the K best complete pools
    of each row's sequence (rows 0 .. total_pools - 1), then its incomplete pool's tokens (rows
    total_pools + s), ascending, -1 suffix."""
    lib = load_library()
    _need(q_idx, "q_idx", torch.bfloat16, 3)
    dev = q_idx.device
    _need(k_pool, "k_pool", torch.bfloat16, 2, dev)
    _need(head_weights, "head_weights", torch.float32, 2, dev)
    T, Hi, Di = q_idx.shape
    W = int(K) + meta.pool - 1
    if topk_idx is None:
        topk_idx = torch.empty(T, W, dtype=torch.int32, device=dev)
    if topk_len is None:
        topk_len = torch.empty(T, dtype=torch.int32, device=dev)
    need = int(lib.dsa_kpool_topk_workspace_size(T, int(K)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _check(lib.dsa_kpool_topk(_ptr(q_idx), _ptr(k_pool), _ptr(head_weights), _ptr(meta.pool_start),
                              _ptr(meta.n_pools), _ptr(meta.tail_start), T, meta.total_pools, Hi, Di, int(K),
                              meta.pool, _ptr(topk_idx), _ptr(topk_len), _ptr(workspace), workspace.numel(),
                              _stream(dev)), "dsa_kpool_topk")
    return topk_idx, topk_len


def dsa_kpool_unpool_grad(dcat: torch.Tensor, meta: KPoolMeta, dx=None):
    """Token key gradient fp32 [T, D] from the gradient of the attended rows fp32 [total_pools + T, D]."""
    lib = load_library()
    _need(dcat, "dcat", torch.float32, 2)
    dev = dcat.device
    D = dcat.shape[1]
    T = meta.total_tokens
    if dx is None:
        dx = torch.empty(T, D, dtype=torch.float32, device=dev)
    _need(dx, "dx", torch.float32, 2, dev)
    _check(lib.dsa_kpool_unpool_grad(_ptr(dcat), T, D, _ptr(meta.cu_seqlens), _ptr(meta.pool_cu), meta.num_seqs,
                                     meta.pool, meta.total_pools, _ptr(dx), _stream(dev)), "dsa_kpool_unpool_grad")
    return dx


def dsa_sparse_mla_fwd(q, kv, topk_idx, softmax_scale: float, topk_len=None, out=None, lse=None,
                       workspace=None, Dv: int = 512, out_lo=None, attn_sink=None):
    """Sparse MLA forward -> (out bf16 [T,H,Dv], lse fp32 [T,H]), or (out, lse, out_lo) when
    out_lo is a tensor or True (the bf16 rounding residual of out, for an exact backward D).
    kv may be [T_k, Dqk] or [T_k, 1, Dqk]; attn_sink: fp32 [H] per-head sink logits or None."""
    lib = load_library()
    _need(q, "q", torch.bfloat16, 3)
    dev = q.device
    if kv.dim() == 3:
        kv = kv.reshape(kv.shape[0], kv.shape[2])
    _need(kv, "kv", torch.bfloat16, 2, dev)
    if topk_idx.dim() == 3:
        topk_idx = topk_idx.reshape(topk_idx.shape[0], topk_idx.shape[2])
    _need(topk_idx, "topk_idx", torch.int32, 2, dev)
    if topk_len is not None:
        _need(topk_len, "topk_len", torch.int32, 1, dev)
    T, H, Dqk = q.shape
    K = topk_idx.shape[1]
    if attn_sink is not None:
        _need(attn_sink, "attn_sink", torch.float32, 1, dev)
        if attn_sink.numel() != H:
            raise ValueError(f"attn_sink must have H = {H} entries")
    if out is None:
        out = torch.empty(T, H, Dv, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(T, H, dtype=torch.float32, device=dev)
    want_lo = out_lo is not None and out_lo is not False
    if out_lo is True:
        out_lo = torch.empty(T, H, Dv, dtype=torch.bfloat16, device=dev)
    lo = out_lo if want_lo else None
    ws, wsb = _workspace("fwd", T, H, dev, workspace)
    _check(lib.dsa_sparse_mla_fwd(_ptr(q), _ptr(kv), _ptr(topk_idx), _ptr(topk_len), T, kv.shape[0], H, Dqk, Dv,
                                  K, float(softmax_scale), _ptr(attn_sink), _ptr(out), _ptr(lo), _ptr(lse), _ptr(ws),
                                  wsb, _stream(dev)),
           "dsa_sparse_mla_fwd")
    return (out, lse, lo) if want_lo else (out, lse)


def dsa_sparse_mla_bwd(q, kv, topk_idx, softmax_scale: float, out, lse, dout, topk_len=None, dq=None,
                       dkv_accum=None, accumulate: bool = False, dkv_bf16=None, workspace=None, out_lo=None,
                       attn_sink=None, d_sink=None, attn_prob=None):
    """Sparse MLA backward -> (dq bf16 [T,H,Dqk], dkv_accum fp32 [T_k,Dqk], dkv_bf16 or None), and
    d_sink fp32 [H] as a fourth result when attn_sink is given (d_sink: an existing tensor to fill,
    or to add to with accumulate=True).
    out_lo: the forward's residual of O (D then uses the fp32 output).
    attn_prob: fp32 [T, K] tensor (or True to allocate one) that receives the head-averaged
    attention probability of every slot; it is then returned as the last result."""
    lib = load_library()
    _need(q, "q", torch.bfloat16, 3)
    dev = q.device
    if kv.dim() == 3:
        kv = kv.reshape(kv.shape[0], kv.shape[2])
    _need(kv, "kv", torch.bfloat16, 2, dev)
    if topk_idx.dim() == 3:
        topk_idx = topk_idx.reshape(topk_idx.shape[0], topk_idx.shape[2])
    _need(topk_idx, "topk_idx", torch.int32, 2, dev)
    _need(out, "out", torch.bfloat16, 3, dev)
    _need(lse, "lse", torch.float32, 2, dev)
    _need(dout, "dout", torch.bfloat16, 3, dev)
    if topk_len is not None:
        _need(topk_len, "topk_len", torch.int32, 1, dev)
    if out_lo is not None:
        _need(out_lo, "out_lo", torch.bfloat16, 3, dev)
    T, H, Dqk = q.shape
    Dv = out.shape[2]
    K = topk_idx.shape[1]
    Tk = kv.shape[0]
    if dq is None:
        dq = torch.empty(T, H, Dqk, dtype=torch.bfloat16, device=dev)
    if dkv_accum is None:
        if accumulate:
            raise ValueError("accumulate=True needs an existing dkv_accum")
        dkv_accum = torch.empty(Tk, Dqk, dtype=torch.float32, device=dev)
    _need(dkv_accum, "dkv_accum", torch.float32, 2, dev)
    if attn_sink is not None:
        _need(attn_sink, "attn_sink", torch.float32, 1, dev)
        if d_sink is None:
            if accumulate:
                raise ValueError("accumulate=True needs an existing d_sink")
            d_sink = torch.empty(H, dtype=torch.float32, device=dev)
        _need(d_sink, "d_sink", torch.float32, 1, dev)
    want_prob = attn_prob is not None and attn_prob is not False
    if attn_prob is True:
        attn_prob = torch.empty(T, K, dtype=torch.float32, device=dev)
    if want_prob:
        _need(attn_prob, "attn_prob", torch.float32, 2, dev)
    ws, wsb = _workspace("bwd", T, H, dev, workspace, K)
    _check(lib.dsa_sparse_mla_bwd(_ptr(q), _ptr(kv), _ptr(topk_idx), _ptr(topk_len), T, Tk, H, Dqk, Dv, K,
                                  float(softmax_scale), _ptr(attn_sink), _ptr(out), _ptr(out_lo), _ptr(lse),
                                  _ptr(dout), _ptr(dq), _ptr(dkv_accum), _ptr(d_sink),
                                  _ptr(attn_prob if want_prob else None), 1 if accumulate else 0, _ptr(dkv_bf16),
                                  _ptr(ws), wsb, _stream(dev)),
           "dsa_sparse_mla_bwd")
    res = (dq, dkv_accum, dkv_bf16) if attn_sink is None else (dq, dkv_accum, dkv_bf16, d_sink)
    return res + (attn_prob,) if want_prob else res


def dsa_sparse_mla_bwd_noalloc(q, kv, topk_idx, softmax_scale: float, out, lse, dout, topk_len=None, dq=None,
                               dkv_accum=None, accumulate: bool = False, dkv_bf16=None, out_lo=None):
    """dsa_sparse_mla_bwd with the library's built-in scratch instead of a workspace (for callers
    that cannot allocate device memory; see include/dsa.h) -> (dq, dkv_accum, dkv_bf16).
    Output tensors the caller does not pass are allocated here by torch, as in the other calls."""
    lib = load_library()
    _need(q, "q", torch.bfloat16, 3)
    dev = q.device
    if kv.dim() == 3:
        kv = kv.reshape(kv.shape[0], kv.shape[2])
    _need(kv, "kv", torch.bfloat16, 2, dev)
    _need(topk_idx, "topk_idx", torch.int32, 2, dev)
    _need(out, "out", torch.bfloat16, 3, dev)
    _need(lse, "lse", torch.float32, 2, dev)
    _need(dout, "dout", torch.bfloat16, 3, dev)
    if topk_len is not None:
        _need(topk_len, "topk_len", torch.int32, 1, dev)
    if out_lo is not None:
        _need(out_lo, "out_lo", torch.bfloat16, 3, dev)
    T, H, Dqk = q.shape
    Tk = kv.shape[0]
    if dq is None:
        dq = torch.empty(T, H, Dqk, dtype=torch.bfloat16, device=dev)
    if dkv_accum is None:
        if accumulate:
            raise ValueError("accumulate=True needs an existing dkv_accum")
        dkv_accum = torch.empty(Tk, Dqk, dtype=torch.float32, device=dev)
    _need(dkv_accum, "dkv_accum", torch.float32, 2, dev)
    _check(lib.dsa_sparse_mla_bwd_noalloc(_ptr(q), _ptr(kv), _ptr(topk_idx), _ptr(topk_len), T, Tk, H, Dqk,
                                          out.shape[2], topk_idx.shape[1], float(softmax_scale), None, _ptr(out),
                                          _ptr(out_lo), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dkv_accum), None, None,
                                          1 if accumulate else 0, _ptr(dkv_bf16), _stream(dev)),
           "dsa_sparse_mla_bwd_noalloc")
    return dq, dkv_accum, dkv_bf16


def dsa_sparse_mla_bwd_noalloc_read_status(device=None) -> int:
    """Synchronise the current stream, read and clear the no-alloc backward's device error word."""
    lib = load_library()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    st = ctypes.c_int32(0)
    _check(lib.dsa_sparse_mla_bwd_noalloc_read_status(_stream(dev), ctypes.byref(st)),
           "dsa_sparse_mla_bwd_noalloc_read_status")
    return st.value


# ---------------------------------------------------------------------------------------------------------------
# The serving step.  These calls may come every few microseconds, so their checks are short: one pass over a tensor's
# attributes, raw pointers, and a device switch only when the tensors live on another device than the current one.
# ---------------------------------------------------------------------------------------------------------------
_NORMS = {"none": 0, "rms": 1, "layer": 2}


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same without the Stream object around it, where torch has it (a third of a short call's time)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def paged_workspace_size(kind: str, a: int = 0, b: int = 0) -> int:
    """Workspace bytes of the serving calls: ("slots"), ("norm_rope_fwd"), ("norm_rope_bwd", rows, norm_dim),
    ("mla", N, H), ("topk", N, max_len), ("quantize"), ("dequantize") or ("mla_quant", N, H).  The first 256 hold the error word, which the calls set and never
    clear: a workspace is made zeroed (torch.zeros), and dsa_read_device_status clears it."""
    lib = load_library()
    if kind in ("slots", "norm_rope_fwd", "quantize", "dequantize"):
        return 256
    if kind == "norm_rope_bwd":
        return int(lib.dsa_norm_rope_bwd_workspace_size(int(b)))
    if kind == "mla":
        return int(lib.dsa_paged_mla_workspace_size())
    if kind == "mla_quant":
        return int(lib.dsa_paged_mla_quant_workspace_size())
    if kind == "topk":
        return int(lib.dsa_paged_indexer_topk_workspace_size(int(a), int(b)))
    raise ValueError(f"unknown workspace kind {kind!r}")


def _dense(t, name, dtype, shape, dev):
    """Data pointer of a contiguous tensor of this type, shape (None: any extent) and device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous() and \
            (dev is None or t.device == dev):
        s = t.shape
        if len(s) == len(shape):
            for n, m in zip(shape, s):
                if n is not None and n != m:
                    break
            else:
                return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have shape {tuple('any' if n is None else n for n in shape)}, got {tuple(t.shape)}")


def _scratch(workspace, need, dev):
    """(workspace, pointer, bytes): the caller's uint8 tensor, or one of `need` bytes."""
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not isinstance(workspace, torch.Tensor) or workspace.dtype is not torch.uint8 or workspace.device != dev:
        raise ValueError(f"workspace must be a uint8 tensor on {dev}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel()


def _call(fn, where, dev, *args):
    """The library call on the tensors' device and its current stream."""
    index = dev.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(index))
    else:
        status = fn(*args, _raw_stream(index))
    if status != DSA_OK:
        _check(status, where)


def dsa_paged_slots(seq_lens, block_table, free_pages, page_size: int, new_lens=None, N: int | None = None,
                    workspace=None):
    """Pages and cache rows of a step's new tokens -> (slot_map int32 [N], positions int32 [N], cu_new int32 [B+1],
    seq_lens_out int32 [B], pages_taken int32 [1]); block_table int32 [B, max_pages] gets the fresh pages, taken
    from free_pages int32 [F] in request order.  new_lens: int32 [B], or None for one token each.  N: entries of
    slot_map and positions (at least the new tokens; -1 beyond them), required with new_lens.  A step that does not fit
    (DSA_ERR_CAPACITY) gives -1 everywhere and cu_new of zeros.  workspace: uint8 [paged_workspace_size("slots")], zeroed
    once, where errors stay until dsa_read_device_status reads them; None: one that is dropped, and the error with it."""
    lib = _lib or load_library()
    p_len = _dense(seq_lens, "seq_lens", torch.int32, (None,), None)
    dev = seq_lens.device
    B = seq_lens.shape[0]
    p_tab = _dense(block_table, "block_table", torch.int32, (B, None), dev)
    p_free = _dense(free_pages, "free_pages", torch.int32, (None,), dev)
    p_new = None if new_lens is None else _dense(new_lens, "new_lens", torch.int32, (B,), dev)
    if N is None:
        if new_lens is not None:
            raise ValueError("N (entries of slot_map and positions) must be given with new_lens")
        N = B
    N = int(N)
    if N < 0:
        raise ValueError("N must be >= 0")
    ws, p_ws, wsb = _scratch(workspace, 256, dev)
    slot_map, positions, cu_new, seq_lens_out, taken = [torch.empty(n, dtype=torch.int32, device=dev)
                                                        for n in (N, N, B + 1, B, 1)]
    _call(lib.dsa_paged_slots, "dsa_paged_slots", dev, p_len, p_new, B, N, int(page_size), block_table.shape[1], p_free,
          free_pages.shape[0], p_tab, seq_lens_out.data_ptr(), cu_new.data_ptr(), slot_map.data_ptr(),
          positions.data_ptr(), taken.data_ptr(), p_ws, wsb)
    return slot_map, positions, cu_new, seq_lens_out, taken


def _rows_of(t, name, dev):
    """(pointer, token stride, head stride, T, H, D) of bf16 rows [T, D] or [T, H, D] with contiguous channels."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    s, st = t.shape, t.stride()
    if len(s) not in (2, 3):
        raise ValueError(f"{name} must be [T, D] or [T, H, D], got shape {tuple(s)}")
    if s[-1] > 1 and st[-1] != 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    return t.data_ptr(), st[0], (st[1] if len(s) == 3 else 0), s[0], (s[1] if len(s) == 3 else 1), s[-1]


def _norm_rope_args(dev, T, D, inv_freq, positions, norm, norm_dim, weight, bias, rope_start):
    if norm not in _NORMS:
        raise ValueError(f"norm must be one of {tuple(_NORMS)}, got {norm!r}")
    kind = _NORMS[norm]
    n = (D if kind else 0) if norm_dim is None else int(norm_dim)
    p_w = None if weight is None else _dense(weight, "weight", torch.float32, (n,), dev)
    p_b = None if bias is None else _dense(bias, "bias", torch.float32, (n,), dev)
    R = 0
    p_f = p_pos = None
    if inv_freq is not None:
        p_f = _dense(inv_freq, "inv_freq", torch.float32, (None,), dev)
        R = 2 * inv_freq.shape[0]
        if positions is None:
            raise ValueError("a rotation needs positions")
        p_pos = _dense(positions, "positions", torch.int32, (T,), dev)
    return kind, n, p_w, p_b, (D - R if rope_start is None else int(rope_start)), R, p_pos, p_f


def dsa_norm_rope_fwd(x, inv_freq=None, positions=None, norm: str = "none", norm_dim: int | None = None, weight=None,
                      bias=None, eps: float = 1e-6, rope_start: int | None = None, interleaved: bool = False,
                      rope_scale: float = 1.0, out=None, out_rows=None, workspace=None):
    """Norm of the first norm_dim channels (default: all) and rotation of 2 * len(inv_freq) channels from rope_start
    (default: the last ones) of bf16 rows x [T, D] or [T, H, D], any strides with contiguous channels -> out, bf16 of
    x's shape (out may be x).  norm: "none", "rms" or "layer"; weight, bias: fp32 [norm_dim]; positions: int32 [T].
    out_rows: int32 [T], the row of `out` that each token goes to (-1: none; a row named twice gets each channel from one of
    the two results); out is then a cache of rows [rows, D], [rows, H, D] or, for x [T, D], pages [num_pages, page_size, D].
    workspace: uint8 [paged_workspace_size("norm_rope_fwd")], zeroed once, where errors (rows outside the cache) stay until
    dsa_read_device_status reads them; None: one that is dropped, and the error with it."""
    lib = _lib or load_library()
    p_x, xt, xh, T, H, D = _rows_of(x, "x", None)
    dev = x.device
    kind, n, p_w, p_b, r0, R, p_pos, p_f = _norm_rope_args(dev, T, D, inv_freq, positions, norm, norm_dim, weight, bias,
                                                           rope_start)
    p_rows, rows = None, 0
    if out_rows is not None:
        if out is None:
            raise ValueError("out_rows needs the cache to write to (out)")
        p_rows = _dense(out_rows, "out_rows", torch.int32, (T,), dev)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=dev)
    cache = out
    if p_rows is not None and x.dim() == 2 and out.dim() == 3:  # pages of rows
        if not out.is_contiguous():
            raise ValueError("a paged cache must be contiguous")
        cache = out.view(-1, out.shape[2])
    p_o, ot, oh, oT, oH, oD = _rows_of(cache, "out", dev)
    if (oH, oD) != (H, D) or (p_rows is None and oT != T):
        raise ValueError(f"out has rows of shape {(oH, oD)} (T = {oT}), x of {(H, D)} (T = {T})")
    if p_rows is not None:
        rows = oT
    ws, p_ws, wsb = _scratch(workspace, 256, dev)
    _call(lib.dsa_norm_rope_fwd, "dsa_norm_rope_fwd", dev, p_x, xt, xh, T, H, D, kind, n, p_w, p_b, eps, r0, R,
          1 if interleaved else 0, p_pos, p_f, rope_scale, p_o, ot, oh, p_rows, rows, p_ws, wsb)
    return out


def dsa_norm_rope_bwd(dout, x=None, inv_freq=None, positions=None, norm: str = "none", norm_dim: int | None = None,
                      weight=None, eps: float = 1e-6, rope_start: int | None = None, interleaved: bool = False,
                      rope_scale: float = 1.0, with_bias: bool = False, dx=None, dweight=None, dbias=None,
                      accumulate: bool = False, workspace=None):
    """Gradient of dsa_norm_rope_fwd -> (dx bf16 of dout's shape, dweight fp32 [norm_dim] or None, dbias fp32
    [norm_dim] or None).  With a norm, x is the forward's input and dweight is always formed; with_bias (layer norm)
    forms dbias too.  accumulate: add to the given dweight / dbias.  dx may be dout or x.  workspace: uint8
    [paged_workspace_size("norm_rope_bwd", rows, norm_dim)]; this call has no errors for dsa_read_device_status."""
    lib = _lib or load_library()
    p_g, gt, gh, T, H, D = _rows_of(dout, "dout", None)
    dev = dout.device
    kind, n, p_w, _, r0, R, p_pos, p_f = _norm_rope_args(dev, T, D, inv_freq, positions, norm, norm_dim, weight, None,
                                                         rope_start)
    p_x = xt = xh = 0
    if kind:
        p_x, xt, xh, xT, xH, xD = _rows_of(x, "x", dev)
        if (xT, xH, xD) != (T, H, D):
            raise ValueError(f"x must have the shape of dout, got {tuple(x.shape)} and {tuple(dout.shape)}")
        if with_bias and kind != 2:
            raise ValueError("only the layer norm has a bias")
        if accumulate and (dweight is None or (with_bias and dbias is None)):
            raise ValueError("accumulate=True needs existing dweight and dbias")
        if dweight is None:
            dweight = torch.empty(n, dtype=torch.float32, device=dev)
        if with_bias and dbias is None:
            dbias = torch.empty(n, dtype=torch.float32, device=dev)
    elif dweight is not None or dbias is not None or with_bias:
        raise ValueError("dweight and dbias belong to a norm")
    p_dw = None if dweight is None else _dense(dweight, "dweight", torch.float32, (n,), dev)
    p_db = None if dbias is None else _dense(dbias, "dbias", torch.float32, (n,), dev)
    if dx is None:
        dx = torch.empty(dout.shape, dtype=torch.bfloat16, device=dev)
    p_d, dt, dh, dT, dH, dD = _rows_of(dx, "dx", dev)
    if (dT, dH, dD) != (T, H, D):
        raise ValueError(f"dx must have the shape of dout, got {tuple(dx.shape)} and {tuple(dout.shape)}")
    ws, p_ws, wsb = _scratch(workspace, 256 if workspace is not None else paged_workspace_size("norm_rope_bwd", 0, n), dev)
    _call(lib.dsa_norm_rope_bwd, "dsa_norm_rope_bwd", dev, p_g, gt, gh, p_x or None, xt, xh, T, H, D, kind, n, p_w, eps,
          r0, R, 1 if interleaved else 0, p_pos, p_f, rope_scale, p_d, dt, dh, p_dw, p_db, 1 if accumulate else 0,
          p_ws, wsb)
    return dx, dweight, dbias


def dsa_rope_frequencies(rope_dim: int, base: float = 10000.0, factor: float = 1.0, original_context: int = 4096,
                         beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Inverse frequencies of a rotation of rope_dim channels, scaled by parts for a context stretched by `factor`
    -> (inv_freq fp32 [rope_dim / 2] on `device` (default: the current CUDA device), rope_scale)."""
    lib = load_library()
    host = torch.empty(max(0, int(rope_dim) // 2), dtype=torch.float32)
    scale = ctypes.c_float(1.0)
    _check(lib.dsa_rope_frequencies(int(rope_dim), float(base), float(factor), int(original_context), float(beta_fast),
                                    float(beta_slow), _ptr(host), ctypes.byref(scale)), "dsa_rope_frequencies")
    return host.to("cuda" if device is None else device), scale.value


def _paged(cache, D, block_table, seq_lens, cu_q, N, dev, dtype=torch.bfloat16):
    """Pointers and sizes of a paged cache: (cache, table, lengths, cu_q, B, num_pages, page_size, max_pages)."""
    p_len = _dense(seq_lens, "seq_lens", torch.int32, (None,), dev)
    B = seq_lens.shape[0]
    p_tab = _dense(block_table, "block_table", torch.int32, (B, None), dev)
    p_cache = _dense(cache, "cache", dtype, (None, None, D), dev)
    p_cu = None
    if cu_q is not None:
        p_cu = _dense(cu_q, "cu_q", torch.int32, (B + 1,), dev)
    elif N != B:
        raise ValueError(f"without cu_q every request has one token: {N} tokens, {B} requests")
    return p_cache, p_tab, p_len, p_cu, B, cache.shape[0], cache.shape[1], block_table.shape[1]


def _lists(topk_idx, topk_len, N, dev):
    """(K, pointer to the lists, pointer to their lengths), or (0, None, None) without lists."""
    if topk_idx is None:
        if topk_len is not None:
            raise ValueError("topk_len needs topk_idx")
        return 0, None, None
    p_idx = _dense(topk_idx, "topk_idx", torch.int32, (N, None), dev)
    K = topk_idx.shape[1]
    if K == 0:  # (an array without entries has no address: the library would take it for no lists at all)
        raise ValueError("topk_idx must have a column at least (an entry of -1 names no position)")
    return K, p_idx, None if topk_len is None else _dense(topk_len, "topk_len", torch.int32, (N,), dev)


def dsa_paged_mla(q, cache, block_table, seq_lens, softmax_scale: float, cu_q=None, topk_idx=None, topk_len=None,
                  attn_sink=None, out=None, lse=None, workspace=None, Dv: int = 512):
    """Attention of new tokens over a paged latent cache -> (out bf16 [N,H,Dv], lse fp32 [N,H]).  q bf16 [N,H,Dqk];
    cache bf16 [num_pages, page_size, Dqk]; block_table int32 [B, max_pages]; seq_lens int32 [B], the new tokens
    included; cu_q int32 [B+1], each request's tokens (None: one each).  topk_idx int32 [N,K] (with topk_len
    int32 [N] or None): attend only to these positions.  attn_sink: fp32 [H] or None.  workspace: uint8
    [paged_workspace_size("mla", N, H)], zeroed once, where errors (bad pages and positions, waits that ran out) stay until
    dsa_read_device_status reads them; None: one that is dropped, and the error with it."""
    lib = _lib or load_library()
    p_q = _dense(q, "q", torch.bfloat16, (None, None, None), None)
    dev = q.device
    N, H, D = q.shape
    p_cache, p_tab, p_len, p_cu, B, pages, page, width = _paged(cache, D, block_table, seq_lens, cu_q, N, dev)
    K, p_idx, p_tl = _lists(topk_idx, topk_len, N, dev)
    p_sink = None if attn_sink is None else _dense(attn_sink, "attn_sink", torch.float32, (H,), dev)
    if out is None:
        out = torch.empty(N, H, Dv, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(N, H, dtype=torch.float32, device=dev)
    p_out = _dense(out, "out", torch.bfloat16, (N, H, Dv), dev)
    p_lse = _dense(lse, "lse", torch.float32, (N, H), dev)
    ws, p_ws, wsb = _scratch(workspace, 0 if workspace is not None else paged_workspace_size("mla"), dev)
    _call(lib.dsa_paged_mla, "dsa_paged_mla", dev, p_q, p_cache, p_tab, p_len, p_cu, p_idx, p_tl, N, B, H, D, Dv, K,
          pages, page, width, softmax_scale, p_sink, p_out, p_lse, p_ws, wsb)
    return out, lse


@functools.lru_cache(maxsize=64)
def _quant_row_bytes(D: int, quant_dim: int, bits: int) -> int:  # (a property of the format)
    return int((_lib or load_library()).dsa_paged_quant_row_bytes(D, quant_dim, bits))


def paged_quant_row_bytes(D: int, bits: int, quant_dim: int | None = None) -> int:
    """Bytes of a row of D channels in a quantised cache (uint8 [num_pages, page_size, row bytes]) whose first quant_dim
    channels (default: 512, or all of fewer) are held in 8 or 4 bits; the format is described in include/dsa.h."""
    q = min(int(D), 512) if quant_dim is None else int(quant_dim)
    n = _quant_row_bytes(int(D), q, int(bits))
    if n == 0:
        raise ValueError(f"no such rows: D = {D}, quant_dim = {q}, bits = {bits} (bits 8 or 4, quant_dim a multiple of 64, "
                         "D <= 1024, the other channels a multiple of 8)")
    return n


def dsa_paged_quantize(x, cache, bits: int, quant_dim: int | None = None, out_rows=None, workspace=None):
    """Rows of bf16 x [T, D] (any token stride, contiguous channels), quantised as they are written to a cache of 8 or 4
    bits -> cache, uint8 [rows, row bytes] or [num_pages, page_size, row bytes] with row bytes of paged_quant_row_bytes(D,
    bits, quant_dim).  quant_dim: so many of the first channels are quantised (default: 512, or all of fewer), the others
    stay bf16.  out_rows: int32 [T], the cache row of each token (-1: none; a row named twice holds bytes of both results),
    e.g. the slots of dsa_paged_slots; None: row t.  A row whose channels are not all finite reads back as NaN.
    workspace: uint8 [paged_workspace_size("quantize")], zeroed once, where errors (rows outside the cache) stay until
    dsa_read_device_status reads them; None: one that is dropped, and the error with it."""
    lib = _lib or load_library()
    p_x, xt, _, T, _, D = _rows_of(x, "x", None)
    if x.dim() != 2:
        raise ValueError(f"x must be [T, D], got shape {tuple(x.shape)}")
    dev = x.device
    q = min(D, 512) if quant_dim is None else int(quant_dim)
    width = paged_quant_row_bytes(D, bits, q)
    paged = isinstance(cache, torch.Tensor) and cache.dim() == 3
    p_c = _dense(cache, "cache", torch.uint8, (None, None, width) if paged else (None, width), dev)
    p_rows = None if out_rows is None else _dense(out_rows, "out_rows", torch.int32, (T,), dev)
    rows = cache.shape[0] * cache.shape[1] if paged else cache.shape[0]
    ws, p_ws, wsb = _scratch(workspace, 256, dev)
    _call(lib.dsa_paged_quantize, "dsa_paged_quantize", dev, p_x, xt, T, D, q, int(bits), p_c, rows, p_rows, p_ws, wsb)
    return cache


def dsa_paged_dequantize(cache, block_table, cu_rows, bits: int, D: int, quant_dim: int | None = None, first=None,
                         N: int | None = None, out=None, workspace=None):
    """Rows of requests read back from a quantised cache (uint8 [num_pages, page_size, row bytes], or [rows, row bytes]
    with pages of one row) -> out bf16 [N, D].  Rows cu_rows[b] .. cu_rows[b+1] - 1 (int32 [B+1]) of out are request b's
    positions first[b], first[b] + 1, ... (int32 [B]; None: from 0) through block_table int32 [B, max_pages].  Rows named
    one by one: pages of one row, and the list as the table of one request.  out: any token stride, its other rows are
    left as they are; None: a new one of N rows (required then).  workspace: uint8 [paged_workspace_size("dequantize")],
    zeroed once, where errors (bad pages and positions; such rows are zeros) stay until dsa_read_device_status reads them;
    None: one that is dropped, and the error with it."""
    lib = _lib or load_library()
    p_cu = _dense(cu_rows, "cu_rows", torch.int32, (None,), None)
    dev = cu_rows.device
    B = cu_rows.shape[0] - 1
    if B < 0:
        raise ValueError("cu_rows must have an entry at least")
    p_tab = _dense(block_table, "block_table", torch.int32, (B, None), dev)
    p_first = None if first is None else _dense(first, "first", torch.int32, (B,), dev)
    D = int(D)
    q = min(D, 512) if quant_dim is None else int(quant_dim)
    width = paged_quant_row_bytes(D, bits, q)
    paged = isinstance(cache, torch.Tensor) and cache.dim() == 3
    p_c = _dense(cache, "cache", torch.uint8, (None, None, width) if paged else (None, width), dev)
    if out is None:
        if N is None:
            raise ValueError("N (rows of the output) must be given without out")
        out = torch.empty(int(N), D, dtype=torch.bfloat16, device=dev)
    p_o, ot, _, n, _, oD = _rows_of(out, "out", dev)
    if out.dim() != 2 or oD != D or (N is not None and n != int(N)):
        raise ValueError(f"out must be [{'N' if N is None else int(N)}, {D}], got shape {tuple(out.shape)}")
    ws, p_ws, wsb = _scratch(workspace, 256, dev)
    _call(lib.dsa_paged_dequantize, "dsa_paged_dequantize", dev, p_c, p_tab, p_first, p_cu, n, B, D, q, int(bits),
          cache.shape[0], cache.shape[1] if paged else 1, block_table.shape[1], p_o, max(ot, D) if n <= 1 else ot, p_ws, wsb)
    return out


def dsa_paged_mla_quant(q, cache, block_table, seq_lens, softmax_scale: float, bits: int, cu_q=None, topk_idx=None,
                        topk_len=None, attn_sink=None, out=None, lse=None, workspace=None, Dv: int = 512):
    """dsa_paged_mla over a cache of latents in 8 or 4 bits (uint8 [num_pages, page_size, paged_quant_row_bytes(Dqk,
    bits)], rows of dsa_paged_quantize) -> (out bf16 [N,H,Dv], lse fp32 [N,H]); the other arguments as there.  workspace:
    uint8 [paged_workspace_size("mla_quant", N, H)], zeroed once, where errors (bad pages and positions, waits that ran out)
    stay until dsa_read_device_status reads them; None: one that is dropped, and the error with it."""
    lib = _lib or load_library()
    p_q = _dense(q, "q", torch.bfloat16, (None, None, None), None)
    dev = q.device
    N, H, D = q.shape
    width = paged_quant_row_bytes(D, bits, 512)
    p_cache, p_tab, p_len, p_cu, B, pages, page, table = _paged(cache, width, block_table, seq_lens, cu_q, N, dev, torch.uint8)
    K, p_idx, p_tl = _lists(topk_idx, topk_len, N, dev)
    p_sink = None if attn_sink is None else _dense(attn_sink, "attn_sink", torch.float32, (H,), dev)
    if out is None:
        out = torch.empty(N, H, Dv, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(N, H, dtype=torch.float32, device=dev)
    p_out = _dense(out, "out", torch.bfloat16, (N, H, Dv), dev)
    p_lse = _dense(lse, "lse", torch.float32, (N, H), dev)
    ws, p_ws, wsb = _scratch(workspace, 0 if workspace is not None else paged_workspace_size("mla_quant"), dev)
    _call(lib.dsa_paged_mla_quant, "dsa_paged_mla_quant", dev, p_q, p_cache, p_tab, p_len, p_cu, p_idx, p_tl, N, B, H, D,
          Dv, int(bits), K, pages, page, table, softmax_scale, p_sink, p_out, p_lse, p_ws, wsb)
    return out, lse


def dsa_paged_indexer_topk(q_idx, k_cache, head_weights, block_table, seq_lens, K: int, cu_q=None,
                           max_len: int | None = None, topk_idx=None, topk_len=None, workspace=None):
    """Top-k selection of new tokens over paged index keys -> (topk_idx int32 [N,K], positions ascending with a -1
    suffix, topk_len int32 [N]): the lists of dsa_paged_mla.  q_idx bf16 [N,Hi,128]; k_cache bf16 [num_pages,
    page_size, 128]; head_weights fp32 [N,Hi]; the rest as dsa_paged_mla.  max_len: no request is longer (default:
    what the table holds), at most 2^30; the workspace is N rows of that many fp32 scores.  workspace: uint8
    [paged_workspace_size("topk", N, max_len)], zeroed once, where errors (bad pages, lengths past max_len, waits that ran
    out) stay until dsa_read_device_status reads them; None: one that is dropped, and the error with it."""
    lib = _lib or load_library()
    p_q = _dense(q_idx, "q_idx", torch.bfloat16, (None, None, None), None)
    dev = q_idx.device
    N, Hi, Di = q_idx.shape
    p_w = _dense(head_weights, "head_weights", torch.float32, (N, Hi), dev)
    p_cache, p_tab, p_len, p_cu, B, pages, page, width = _paged(k_cache, Di, block_table, seq_lens, cu_q, N, dev)
    K = int(K)
    max_len = min(width * page, 2 ** 30) if max_len is None else int(max_len)
    if topk_idx is None:
        topk_idx = torch.empty(N, K, dtype=torch.int32, device=dev)
    if topk_len is None:
        topk_len = torch.empty(N, dtype=torch.int32, device=dev)
    p_idx = _dense(topk_idx, "topk_idx", torch.int32, (N, K), dev)
    p_tl = _dense(topk_len, "topk_len", torch.int32, (N,), dev)
    ws, p_ws, wsb = _scratch(workspace, 0 if workspace is not None else paged_workspace_size("topk", N, max_len), dev)
    _call(lib.dsa_paged_indexer_topk, "dsa_paged_indexer_topk", dev, p_q, p_cache, p_w, p_tab, p_len, p_cu, N, B, Hi, Di,
          K, pages, page, width, max_len, p_idx, p_tl, p_ws, wsb)
    return topk_idx, topk_len


def dsa_set_wait_limit_cycles(cycles: int) -> int:
    """Cycle limit of the kernels' bounded waits for later launches (negative: the default, 2^31);
    returns the previous limit."""
    return int(load_library().dsa_set_wait_limit_cycles(int(cycles)))


def dsa_read_device_status(workspace: torch.Tensor) -> int:
    """Synchronise the current stream, read and clear the device error word of ``workspace``."""
    lib = load_library()
    st = ctypes.c_int32(0)
    _check(lib.dsa_read_device_status(_ptr(workspace), _stream(workspace.device), ctypes.byref(st)),
           "dsa_read_device_status")
    return st.value
