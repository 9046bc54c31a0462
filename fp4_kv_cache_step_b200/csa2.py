"""Thin Python binding of libcsa2_fp4 (include/csa2.h).

Argument marshalling only: the functions below take torch CUDA tensors, check
their dtype/shape/contiguity, allocate outputs and workspace with torch, and
call the C ABI of the same name on the current torch stream. Every step of the
computation runs in the library's CUDA kernels; there is no fallback. If the
shared library is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa2_fp4.so")

MODE_FULL, MODE_REINDEX, MODE_REUSE = 0, 1, 2
_MODES = {"FULL": MODE_FULL, "REINDEX": MODE_REINDEX, "REUSE": MODE_REUSE}
STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CUDA", 4: "DEVICE_INDEX",
          5: "NONFINITE", 6: "TIMEOUT", 7: "WORKSPACE", 8: "NO_PAGES"}


class Csa2Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("%s (%s)" % (msg, STATUS.get(status, status)))
        self.status = status


class SharedState(ctypes.Structure):
    _fields_ = [("kv_packed", ctypes.c_void_p), ("kv_scale", ctypes.c_void_p),
                ("idx_k", ctypes.c_void_p), ("topk_idx", ctypes.c_void_p),
                ("cand_idx", ctypes.c_void_p), ("C", ctypes.c_int)]


class LayerArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Tq", ctypes.c_int), ("N", ctypes.c_int),
                ("D", ctypes.c_int), ("Hq", ctypes.c_int), ("Hi", ctypes.c_int),
                ("Di", ctypes.c_int), ("K", ctypes.c_int), ("nvalid", ctypes.c_void_p),
                ("q", ctypes.c_void_p), ("idx_q", ctypes.c_void_p), ("idx_w", ctypes.c_void_p),
                ("softmax_scale", ctypes.c_float), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("emit_pool", ctypes.c_int),
                ("use_pool", ctypes.c_int), ("swa_kv", ctypes.c_void_p),
                ("swa_n", ctypes.c_void_p), ("Tw", ctypes.c_int), ("W", ctypes.c_int)]


class PagesStruct(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("table", ctypes.c_void_p), ("len", ctypes.c_void_p),
                ("refs", ctypes.c_void_p), ("P", ctypes.c_int), ("page", ctypes.c_int),
                ("D", ctypes.c_int), ("S", ctypes.c_int), ("M", ctypes.c_int)]


class NormRopeArgs(ctypes.Structure):
    _fields_ = [("D", ctypes.c_int), ("R", ctypes.c_int), ("rot_begin", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("inverse", ctypes.c_int),
                ("rot_scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("turns", ctypes.c_void_p), ("T", ctypes.c_int), ("Hq", ctypes.c_int),
                ("q_norm", ctypes.c_int), ("q_f32", ctypes.c_int), ("q", ctypes.c_void_p),
                ("q_stride", ctypes.c_longlong), ("pos", ctypes.c_void_p),
                ("q_weight", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("E", ctypes.c_int),
                ("kv_norm", ctypes.c_int), ("kv_f32", ctypes.c_int), ("kv", ctypes.c_void_p),
                ("kv_stride", ctypes.c_longlong), ("kv_pos", ctypes.c_void_p),
                ("kv_weight", ctypes.c_void_p), ("seq", ctypes.c_void_p),
                ("entry", ctypes.c_void_p), ("kv_out", ctypes.c_void_p)]


EXPORTS = ("fp4_kv_pack", "fp4_kv_unpack", "csa2_index_score", "csa2_topk",
           "csa2_sparse_attn_workspace_bytes", "csa2_sparse_attn",
           "csa2_layer_step_workspace_bytes", "csa2_layer_step", "csa2_check_device_errors",
           "csa2_last_error", "csa2_sparse_attn_noalloc", "fp4_kv_pack_g16", "fp4_kv_unpack_g16",
           "fp4_kv_append_g16", "csa2_sparse_attn_g16", "csa2_block_pool_workspace_bytes",
           "csa2_block_pool", "csa2_sparse_attn_swa", "fp4_kv_pages_resize",
           "fp4_kv_pages_resize_workspace_bytes", "fp4_kv_pages_fork",
           "fp4_kv_pages_fork_workspace_bytes", "fp4_kv_pages_compact",
           "fp4_kv_pages_compact_workspace_bytes", "csa2_rope_turns", "csa2_qk_norm_rope",
           "csa2_paged_attn", "csa2_paged_attn_workspace_bytes")

_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libcsa2_fp4.so not found at %s: build it with "
                           "`python -m fp4_kv_cache_step_b200.build`" % path)
    L = ctypes.CDLL(path)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.fp4_kv_pack.argtypes = [P, I, I, I, P, P, P]
    L.fp4_kv_unpack.argtypes = [P, P, I, I, I, P, P]
    L.csa2_index_score.argtypes = [P, P, P, I, I, I, I, I, P, P, I, P, P]
    L.csa2_topk.argtypes = [P, I, P, P, I, I, I, P, I, P, P]
    L.csa2_sparse_attn_workspace_bytes.argtypes = [I, I, I, I, I]
    L.csa2_sparse_attn_workspace_bytes.restype = Z
    L.csa2_sparse_attn.argtypes = [P, P, P, P, I, I, I, I, I, I, F, P, P, P, Z, P]
    L.csa2_sparse_attn_noalloc.argtypes = [P, P, P, P, I, I, I, I, I, I, F, P, P, P]
    L.fp4_kv_pack_g16.argtypes = [P, I, I, I, P, P]
    L.fp4_kv_unpack_g16.argtypes = [P, I, I, I, P, P]
    L.fp4_kv_append_g16.argtypes = [P, P, I, I, I, I, P, P]
    L.csa2_sparse_attn_g16.argtypes = [P, P, P, I, I, I, I, I, I, F, P, P, P, Z, P]
    L.csa2_sparse_attn_swa.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, P, P, P, Z,
                                       P]
    L.csa2_block_pool_workspace_bytes.argtypes = [I, I, I, I, I]
    L.csa2_block_pool_workspace_bytes.restype = Z
    L.csa2_block_pool.argtypes = [P, I, P, I, I, I, I, P, P, Z, P]
    L.csa2_layer_step_workspace_bytes.argtypes = [ctypes.POINTER(LayerArgs), I,
                                                  ctypes.POINTER(SharedState)]
    L.csa2_layer_step_workspace_bytes.restype = Z
    L.csa2_layer_step.argtypes = [ctypes.POINTER(LayerArgs), I, ctypes.POINTER(SharedState), P, Z, P]
    G = ctypes.POINTER(PagesStruct)
    L.fp4_kv_pages_resize.argtypes = [G, P, P, I, P, Z, P]
    L.fp4_kv_pages_fork.argtypes = [G, P, P, I, P, Z, P]
    L.fp4_kv_pages_compact.argtypes = [G, P, P, Z, P]
    L.fp4_kv_pages_resize_workspace_bytes.argtypes = [G, I]
    L.fp4_kv_pages_fork_workspace_bytes.argtypes = [G, I]
    L.fp4_kv_pages_compact_workspace_bytes.argtypes = [G]
    L.csa2_rope_turns.argtypes = [I, ctypes.c_double, I, ctypes.c_double, ctypes.c_double,
                                  ctypes.c_double, ctypes.c_double, P]
    L.csa2_qk_norm_rope.argtypes = [ctypes.POINTER(NormRopeArgs), G, P]
    L.csa2_paged_attn.argtypes = [P, G, P, P, P, I, I, I, I, F, P, P, P, Z, P]
    L.csa2_paged_attn_workspace_bytes.argtypes = [G, I, I, I, I]
    for f in ("fp4_kv_pages_resize", "fp4_kv_pages_fork", "fp4_kv_pages_compact",
              "csa2_paged_attn"):
        getattr(L, f + "_workspace_bytes").restype = Z
    L.csa2_check_device_errors.argtypes = [P]
    L.csa2_last_error.argtypes = []
    L.csa2_last_error.restype = ctypes.c_char_p
    for f in ("fp4_kv_pack", "fp4_kv_unpack", "csa2_index_score", "csa2_topk", "csa2_sparse_attn",
              "csa2_layer_step", "csa2_check_device_errors", "csa2_sparse_attn_noalloc",
              "fp4_kv_pack_g16", "fp4_kv_unpack_g16", "fp4_kv_append_g16", "csa2_sparse_attn_g16",
              "csa2_block_pool", "csa2_sparse_attn_swa", "fp4_kv_pages_resize",
              "fp4_kv_pages_fork", "fp4_kv_pages_compact", "csa2_rope_turns", "csa2_qk_norm_rope",
              "csa2_paged_attn"):
        getattr(L, f).restype = I
    _lib = L
    return L


def _check(rc: int, what: str):
    if rc != 0:
        msg = load().csa2_last_error().decode(errors="replace")
        raise Csa2Error(rc, "%s: %s" % (what, msg))


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _want(t, dtype, name, ndim=None):
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dims, got shape %s" % (name, ndim, tuple(t.shape)))


def check_device_errors():
    """Synchronise the current stream and raise if a kernel recorded a data error."""
    _check(load().csa2_check_device_errors(_stream()), "csa2_check_device_errors")


# ------------------------------------------------------------------- FP4 KV
def fp4_kv_pack(kv: torch.Tensor, packed: Optional[torch.Tensor] = None,
                scale: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """kv float32 [B][N][D] -> (packed uint8 [B][N][D/2], scale uint8 [B][N/64][D])."""
    _want(kv, torch.float32, "kv", 3)
    B, N, D = kv.shape
    if packed is None:
        packed = torch.empty((B, N, D // 2), dtype=torch.uint8, device=kv.device)
    if scale is None:
        scale = torch.empty((B, N // 64, D), dtype=torch.uint8, device=kv.device)
    _check(load().fp4_kv_pack(_p(kv), B, N, D, _p(packed), _p(scale), _stream(kv.device)),
           "fp4_kv_pack")
    return packed, scale


def fp4_kv_unpack(packed: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    _want(packed, torch.uint8, "packed", 3)
    _want(scale, torch.uint8, "scale", 3)
    B, N, Dh = packed.shape
    out = torch.empty((B, N, 2 * Dh), dtype=torch.float32, device=packed.device)
    _check(load().fp4_kv_unpack(_p(packed), _p(scale), B, N, 2 * Dh, _p(out),
                                _stream(packed.device)), "fp4_kv_unpack")
    return out


# ------------------------------------------------------------------- FP4 KV, 16-channel scales
def g16_row_bytes(D: int) -> int:
    """Bytes of one entry in the 16-channel layout: D/2 codes, then D/16 scales."""
    return D // 2 + D // 16


def fp4_kv_pack_g16(kv: torch.Tensor, rows: Optional[torch.Tensor] = None) -> torch.Tensor:
    """kv float32 [B][N][D] -> rows uint8 [B][N][D/2 + D/16]."""
    _want(kv, torch.float32, "kv", 3)
    B, N, D = kv.shape
    if rows is None:
        rows = torch.empty((B, N, g16_row_bytes(D)), dtype=torch.uint8, device=kv.device)
    _check(load().fp4_kv_pack_g16(_p(kv), B, N, D, _p(rows), _stream(kv.device)),
           "fp4_kv_pack_g16")
    return rows


def fp4_kv_unpack_g16(rows: torch.Tensor, D: int) -> torch.Tensor:
    _want(rows, torch.uint8, "rows", 3)
    B, N, rb = rows.shape
    if rb != g16_row_bytes(D):
        raise ValueError("rows of %d bytes do not hold D=%d" % (rb, D))
    out = torch.empty((B, N, D), dtype=torch.float32, device=rows.device)
    _check(load().fp4_kv_unpack_g16(_p(rows), B, N, D, _p(out), _stream(rows.device)),
           "fp4_kv_unpack_g16")
    return out


def fp4_kv_append_g16(rows: torch.Tensor, kv_new: torch.Tensor, pos: torch.Tensor) -> torch.Tensor:
    """Quantise kv_new float32 [B][T][D] into rows[b][pos[b][t]] in place."""
    _want(rows, torch.uint8, "rows", 3)
    _want(kv_new, torch.float32, "kv_new", 3)
    _want(pos, torch.int32, "pos", 2)
    B, T, D = kv_new.shape
    N = rows.shape[1]
    _check(load().fp4_kv_append_g16(_p(kv_new), _p(pos), B, T, N, D, _p(rows),
                                    _stream(rows.device)), "fp4_kv_append_g16")
    return rows


# ------------------------------------------------------------------- indexer
def csa2_index_score(idx_q: torch.Tensor, idx_w: torch.Tensor, idx_k: torch.Tensor,
                     nvalid: Optional[torch.Tensor] = None, cand: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """idx_q uint8 (E4M3) [B][Tq][Hi][Di], idx_w float32 [B][Tq][Hi], idx_k uint8 [B][N][Di]
    -> scores float32 [B][Tq][N] (or [B][Tq][C] with a candidate pool)."""
    _want(idx_q, torch.uint8, "idx_q", 4)
    _want(idx_w, torch.float32, "idx_w", 3)
    _want(idx_k, torch.uint8, "idx_k", 3)
    B, Tq, Hi, Di = idx_q.shape
    N = idx_k.shape[1]
    C = 0
    if cand is not None:
        _want(cand, torch.int32, "cand", 3)
        C = cand.shape[-1]
    elif nvalid is not None:
        _want(nvalid, torch.int32, "nvalid", 2)
    if out is None:
        out = torch.empty((B, Tq, C if cand is not None else N), dtype=torch.float32,
                          device=idx_q.device)
    _check(load().csa2_index_score(_p(idx_q), _p(idx_w), _p(idx_k), B, Tq, N, Hi, Di, _p(nvalid),
                                   _p(cand), C, _p(out), _stream(idx_q.device)), "csa2_index_score")
    return out


def csa2_topk(scores: torch.Tensor, K: int, nvalid: Optional[torch.Tensor] = None,
              cand: Optional[torch.Tensor] = None, Cout: int = 0,
              out: Optional[torch.Tensor] = None, cand_out: Optional[torch.Tensor] = None):
    """scores float32 [B][Tq][ld] -> topk int32 [B][Tq][K] (and the top-Cout pool)."""
    _want(scores, torch.float32, "scores", 3)
    B, Tq, ld = scores.shape
    if out is None:
        out = torch.empty((B, Tq, K), dtype=torch.int32, device=scores.device)
    if Cout and cand_out is None:
        cand_out = torch.empty((B, Tq, Cout), dtype=torch.int32, device=scores.device)
    _check(load().csa2_topk(_p(scores), ld, _p(nvalid), _p(cand), B, Tq, K, _p(out), int(Cout),
                            _p(cand_out), _stream(scores.device)), "csa2_topk")
    return (out, cand_out) if Cout else out


def csa2_block_pool(scores: torch.Tensor, nvalid: torch.Tensor, nblocks: int, block: int = 8,
                    out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scores float32 [B][Tq][ld] -> the blockwise pool int32 [B][Tq][nblocks * block]."""
    _want(scores, torch.float32, "scores", 3)
    _want(nvalid, torch.int32, "nvalid", 2)
    B, Tq, ld = scores.shape
    L = load()
    if out is None:
        out = torch.empty((B, Tq, nblocks * block), dtype=torch.int32, device=scores.device)
    need = L.csa2_block_pool_workspace_bytes(B, Tq, ld, block, nblocks)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=scores.device)
    _check(L.csa2_block_pool(_p(scores), ld, _p(nvalid), B, Tq, int(block), int(nblocks), _p(out),
                             _p(workspace) if need else None, need, _stream(scores.device)),
           "csa2_block_pool")
    return out


# ------------------------------------------------------------------- attention
def csa2_sparse_attn(q: torch.Tensor, kv_packed: torch.Tensor, kv_scale: torch.Tensor,
                     topk_idx: torch.Tensor, softmax_scale: float, want_lse: bool = True,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None):
    """q bf16 [B][Tq][Hq][D] -> (out bf16 [B][Tq][Hq][D], lse float32 [B][Tq][Hq] or None)."""
    _want(q, torch.bfloat16, "q", 4)
    _want(topk_idx, torch.int32, "topk_idx", 3)
    B, Tq, Hq, D = q.shape
    N = kv_packed.shape[1]
    K = topk_idx.shape[-1]
    L = load()
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((B, Tq, Hq), dtype=torch.float32, device=q.device)
    need = L.csa2_sparse_attn_workspace_bytes(B, Tq, Hq, D, K)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(L.csa2_sparse_attn(_p(q), _p(kv_packed), _p(kv_scale), _p(topk_idx), B, Tq, Hq, D, N, K,
                              float(softmax_scale), _p(out), _p(lse if want_lse else None),
                              _p(workspace) if need else None, need, _stream(q.device)),
           "csa2_sparse_attn")
    return out, (lse if want_lse else None)


def csa2_sparse_attn_g16(q: torch.Tensor, kv_rows: torch.Tensor, topk_idx: torch.Tensor,
                         softmax_scale: float, want_lse: bool = True,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None):
    """csa2_sparse_attn over a cache in the 16-channel layout (fp4_kv_pack_g16)."""
    _want(q, torch.bfloat16, "q", 4)
    _want(kv_rows, torch.uint8, "kv_rows", 3)
    _want(topk_idx, torch.int32, "topk_idx", 3)
    B, Tq, Hq, D = q.shape
    N = kv_rows.shape[1]
    K = topk_idx.shape[-1]
    L = load()
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((B, Tq, Hq), dtype=torch.float32, device=q.device)
    need = L.csa2_sparse_attn_workspace_bytes(B, Tq, Hq, D, K)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(L.csa2_sparse_attn_g16(_p(q), _p(kv_rows), _p(topk_idx), B, Tq, Hq, D, N, K,
                                  float(softmax_scale), _p(out), _p(lse if want_lse else None),
                                  _p(workspace) if need else None, need, _stream(q.device)),
           "csa2_sparse_attn_g16")
    return out, (lse if want_lse else None)


SWA_WINDOW = 128   # tokens in the sliding window of every CSA2 layer


def csa2_sparse_attn_swa(q: torch.Tensor, kv_packed: torch.Tensor,
                         kv_scale: Optional[torch.Tensor], topk_idx: torch.Tensor,
                         swa_kv: torch.Tensor, swa_n: torch.Tensor, softmax_scale: float,
                         W: int = SWA_WINDOW, want_lse: bool = True,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None):
    """csa2_sparse_attn plus the sliding-window branch: one softmax over the
    selected rows and the tokens [max(0, n - W), n) of each row's E4M3 window
    memory swa_kv uint8 [B][Tw][D], n = swa_n int32 [B][Tq]. kv_scale None:
    kv_packed is in the 16-channel layout."""
    _want(q, torch.bfloat16, "q", 4)
    _want(topk_idx, torch.int32, "topk_idx", 3)
    _want(swa_kv, torch.uint8, "swa_kv", 3)
    _want(swa_n, torch.int32, "swa_n", 2)
    B, Tq, Hq, D = q.shape
    N = kv_packed.shape[1]
    K = topk_idx.shape[-1]
    Tw = swa_kv.shape[1]
    L = load()
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((B, Tq, Hq), dtype=torch.float32, device=q.device)
    need = L.csa2_sparse_attn_workspace_bytes(B, Tq, Hq, D, K + int(W))
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(L.csa2_sparse_attn_swa(_p(q), _p(kv_packed), _p(kv_scale), _p(topk_idx), _p(swa_kv),
                                  _p(swa_n), B, Tq, Hq, D, N, K, Tw, int(W),
                                  float(softmax_scale), _p(out), _p(lse if want_lse else None),
                                  _p(workspace) if need else None, need, _stream(q.device)),
           "csa2_sparse_attn_swa")
    return out, (lse if want_lse else None)


def csa2_sparse_attn_noalloc(q: torch.Tensor, kv_packed: torch.Tensor, kv_scale: torch.Tensor,
                             topk_idx: torch.Tensor, softmax_scale: float, want_lse: bool = True,
                             out: Optional[torch.Tensor] = None,
                             lse: Optional[torch.Tensor] = None):
    """csa2_sparse_attn for callers that cannot allocate device memory: the
    library's built-in scratch array stands in for the workspace (outputs are
    still the caller's). Calls that overlap on the GPU must be avoided."""
    _want(q, torch.bfloat16, "q", 4)
    _want(topk_idx, torch.int32, "topk_idx", 3)
    B, Tq, Hq, D = q.shape
    N = kv_packed.shape[1]
    K = topk_idx.shape[-1]
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((B, Tq, Hq), dtype=torch.float32, device=q.device)
    _check(load().csa2_sparse_attn_noalloc(_p(q), _p(kv_packed), _p(kv_scale), _p(topk_idx), B, Tq,
                                           Hq, D, N, K, float(softmax_scale), _p(out),
                                           _p(lse if want_lse else None), _stream(q.device)),
           "csa2_sparse_attn_noalloc")
    return out, (lse if want_lse else None)


class Csa2Shared:
    """Buffers one stack of CSA2 layers shares: the FP4 main KV and indexer keys
    a FULL layer built, and the latest top-K (and candidate pool)."""

    def __init__(self, kv_packed, kv_scale, idx_k, topk_idx, cand_idx=None):
        self.kv_packed, self.kv_scale, self.idx_k = kv_packed, kv_scale, idx_k
        self.topk_idx, self.cand_idx = topk_idx, cand_idx

    def c_struct(self) -> SharedState:
        return SharedState(_p(self.kv_packed), _p(self.kv_scale), _p(self.idx_k),
                           _p(self.topk_idx), _p(self.cand_idx),
                           0 if self.cand_idx is None else int(self.cand_idx.shape[-1]))


def layer_args(q, nvalid, out, K, softmax_scale, idx_q=None, idx_w=None, lse=None, N=None,
               emit_pool=False, use_pool=False, swa_kv=None, swa_n=None,
               W=SWA_WINDOW) -> LayerArgs:
    """emit_pool: False/0 none, True/1 the top-C entries, 2 the blockwise pool.
    swa_kv / swa_n: the sliding-window branch (as in csa2_sparse_attn_swa)."""
    B, Tq, Hq, D = q.shape
    Hi = Di = 0
    if idx_q is not None:
        Hi, Di = idx_q.shape[2], idx_q.shape[3]
    Tw = 0 if swa_kv is None else int(swa_kv.shape[1])
    return LayerArgs(B, Tq, int(N), D, Hq, Hi, Di, int(K), _p(nvalid), _p(q), _p(idx_q),
                     _p(idx_w), float(softmax_scale), _p(out), _p(lse), int(emit_pool),
                     int(bool(use_pool)), _p(swa_kv), _p(swa_n), Tw,
                     int(W) if swa_kv is not None else 0)


def csa2_layer_step(mode, args: LayerArgs, shared: Csa2Shared,
                    workspace: Optional[torch.Tensor] = None, device=None) -> torch.Tensor:
    """Run one CSA2 layer in `mode` ("FULL" | "REINDEX" | "REUSE" or 0/1/2)."""
    m = _MODES[mode] if isinstance(mode, str) else int(mode)
    L = load()
    st = shared.c_struct()
    need = L.csa2_layer_step_workspace_bytes(ctypes.byref(args), m, ctypes.byref(st))
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=shared.kv_packed.device)
    _check(L.csa2_layer_step(ctypes.byref(args), m, ctypes.byref(st),
                             _p(workspace) if need else None, need,
                             _stream(shared.kv_packed.device)), "csa2_layer_step")
    return workspace


def layer_step_workspace_bytes(mode, args: LayerArgs, shared: Csa2Shared) -> int:
    m = _MODES[mode] if isinstance(mode, str) else int(mode)
    st = shared.c_struct()
    return int(load().csa2_layer_step_workspace_bytes(ctypes.byref(args), m, ctypes.byref(st)))


# ------------------------------------------------------------------- paged cache
# (The calls below take microseconds on the GPU, so their checks avoid what costs
# as much on the host: device objects, Stream objects, keyword parsing.)
_BF16, _F32, _I32, _I64, _U8 = (torch.bfloat16, torch.float32, torch.int32, torch.int64,
                                torch.uint8)


def _at(t, name, index):
    """A tensor's pointer, if it is on CUDA device `index`."""
    if t.get_device() != index:
        raise ValueError("%s must be on cuda:%d, got %s" % (name, index, t.device))
    return t.data_ptr()


def _vec(t, name, dtype, n, index):
    """A contiguous tensor of n values on CUDA device `index`: its pointer."""
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be contiguous with %d values, got shape %s"
                         % (name, n, tuple(t.shape)))
    if t.get_device() != index:
        raise ValueError("%s must be on cuda:%d, got %s" % (name, index, t.device))
    return t.data_ptr()


def _call(name, index, *args):
    """The C call of that name on the current stream of CUDA device `index`, with
    that device current (a default stream belongs to the current device)."""
    fn = getattr(_lib or load(), name)
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != 0:
        _check(rc, name)


def _scratch(workspace, need, device):
    """(tensor, pointer, bytes) of the caller's workspace, or of a new one."""
    if workspace is None:
        workspace = torch.empty(need, dtype=_U8, device=device)
        return workspace, workspace.data_ptr(), need
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % device)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


class Fp4Pages:
    """A paged FP4 cache (fp4_kv_pages in csa2.h) over the caller's tensors: rows
    uint8 [P][page][D/2 + D/16], table int32 [S][M] (-1: no page), length int32
    [S], refs int32 [P] (0: the page is free). Holds the tensors, nothing else."""

    def __init__(self, rows: torch.Tensor, table: torch.Tensor, length: torch.Tensor,
                 refs: torch.Tensor):
        _want(rows, _U8, "rows", 3)
        _want(table, _I32, "table", 2)
        _want(length, _I32, "length", 1)
        _want(refs, _I32, "refs", 1)
        P, page, rb = rows.shape
        S, M = table.shape
        if rb == 0 or rb % 72 != 0:
            raise ValueError("rows of %d bytes hold no multiple of 128 channels" % rb)
        if length.shape[0] != S or refs.shape[0] != P:
            raise ValueError("length and refs must have S=%d and P=%d values" % (S, P))
        if not rows.is_cuda:
            raise ValueError("expected CUDA tensors")
        self.device, self.index = rows.device, rows.get_device()
        for t, name in ((rows, "rows"), (table, "table"), (length, "length"), (refs, "refs")):
            _at(t, name, self.index)
            if not t.is_contiguous():
                raise ValueError("expected contiguous %s" % name)
        self.rows, self.table, self.length, self.refs = rows, table, length, refs
        self.P, self.page, self.D, self.S, self.M = P, page, rb // 72 * 128, S, M
        self._c = PagesStruct(rows.data_ptr(), table.data_ptr(), length.data_ptr(),
                              refs.data_ptr(), P, page, self.D, S, M)
        self.ref = ctypes.byref(self._c)
        self._sizes = {}

    def workspace_bytes(self, call: str, *shape: int) -> int:
        """Workspace of a paged call for a shape (asked once per shape)."""
        need = self._sizes.get((call, shape))
        if need is None:
            with torch.cuda.device(self.index):
                need = getattr(load(), call + "_workspace_bytes")(self.ref, *shape)
            self._sizes[call, shape] = need
        return need

    @classmethod
    def empty(cls, P: int, page: int, D: int, S: int, M: int, device="cuda") -> "Fp4Pages":
        """A cache of P free pages and S empty slots of up to M pages."""
        return cls(torch.zeros((P, page, g16_row_bytes(D)), dtype=_U8, device=device),
                   torch.full((S, M), -1, dtype=_I32, device=device),
                   torch.zeros(S, dtype=_I32, device=device),
                   torch.zeros(P, dtype=_I32, device=device))


def fp4_kv_pages_resize(pages: Fp4Pages, seq: torch.Tensor, new_len: torch.Tensor,
                        workspace: Optional[torch.Tensor] = None) -> None:
    """Slots seq int32 [n] get new_len int32 [n] entries: pages behind are given
    back, free ones taken lowest first; a shared, partly filled last page that
    grows is copied. Length 0 frees a slot."""
    n, index = seq.numel(), pages.index
    a, b = _vec(seq, "seq", _I32, n, index), _vec(new_len, "new_len", _I32, n, index)
    ws, p, size = _scratch(workspace, pages.workspace_bytes("fp4_kv_pages_resize", n),
                           pages.device)
    _call("fp4_kv_pages_resize", index, pages.ref, a, b, n, p, size)


def fp4_kv_pages_fork(pages: Fp4Pages, src: torch.Tensor, dst: torch.Tensor,
                      workspace: Optional[torch.Tensor] = None) -> None:
    """Slot dst[i] becomes a copy of slot src[i] (int32 [n], at once): the pages
    are shared, what dst[i] held is given back."""
    n, index = src.numel(), pages.index
    a, b = _vec(src, "src", _I32, n, index), _vec(dst, "dst", _I32, n, index)
    ws, p, size = _scratch(workspace, pages.workspace_bytes("fp4_kv_pages_fork", n),
                           pages.device)
    _call("fp4_kv_pages_fork", index, pages.ref, a, b, n, p, size)


def fp4_kv_pages_compact(pages: Fp4Pages, used: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None) -> None:
    """Move the U pages in use to the places [0, U); used int32 [1] receives U."""
    u = None if used is None else _vec(used, "used", _I32, 1, pages.index)
    ws, p, size = _scratch(workspace, pages.workspace_bytes("fp4_kv_pages_compact"),
                           pages.device)
    _call("fp4_kv_pages_compact", pages.index, pages.ref, u, p, size)


# ------------------------------------------------------------------- norm, rotation, append
_ROPE_SCALING = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}


def csa2_rope_turns(R: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                    context: float = 0.0, fast: float = 32.0, slow: float = 1.0,
                    device="cuda") -> torch.Tensor:
    """Rotation frequencies of R channels as int64 [R/2]: the turns per position of
    each pair, times 2^64 (computed on the host, then copied to `device`)."""
    if scaling not in _ROPE_SCALING:
        raise ValueError("scaling must be one of %s" % ", ".join(_ROPE_SCALING))
    turns = torch.empty(max(0, R) // 2, dtype=_I64)
    _check(load().csa2_rope_turns(int(R), float(base), _ROPE_SCALING[scaling], float(factor),
                                  float(context), float(fast), float(slow),
                                  turns.data_ptr() if turns.numel() else None), "csa2_rope_turns")
    return turns.to(device)


# csa2_norm_rope_args, packed in one go (checked against NormRopeArgs below)
_ROPE_PACK = struct.Struct("@5i2fxxxxP4iPqPPPiiixxxxPqPPPPP")
assert _ROPE_PACK.size == ctypes.sizeof(NormRopeArgs)


def csa2_qk_norm_rope(turns: torch.Tensor, rot_begin: int, interleaved: bool = True,
                      inverse: bool = False, rot_scale: float = 1.0, eps: float = 1e-6,
                      q: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None,
                      q_norm: bool = True, q_weight: Optional[torch.Tensor] = None,
                      q_out: Optional[torch.Tensor] = None, kv: Optional[torch.Tensor] = None,
                      kv_pos: Optional[torch.Tensor] = None, kv_norm: bool = True,
                      kv_weight: Optional[torch.Tensor] = None, pages: Optional[Fp4Pages] = None,
                      seq: Optional[torch.Tensor] = None, entry: Optional[torch.Tensor] = None,
                      kv_out: Optional[torch.Tensor] = None):
    """RMS norm and rotary embedding of queries q [T][Hq][D] (bf16 or float32,
    heads contiguous, any token stride) -> q_out bf16, and of entries kv [E][D]
    quantised into row entry[e] of slot seq[e] of `pages` (kv_out: the bf16 values
    that the rows stand for, when given). Either part may be left out. Channels
    [rot_begin, rot_begin + R) turn by pos (kv_pos) int32 times `turns` [R/2]."""
    if q is None and kv is None:
        raise ValueError("nothing to do: give q, kv or both")
    index = (q if q is not None else kv).get_device()
    R2 = turns.numel()
    if turns.dim() != 1:
        raise ValueError("turns must have 1 dim, got shape %s" % (tuple(turns.shape),))
    p_turns = _vec(turns, "turns", _I64, R2, index) if R2 else 0
    D = T = H = q_f32 = q_stride = p_q = p_pos = p_qw = p_qo = 0
    E = kv_f32 = kv_stride = p_kv = p_kp = p_kw = p_seq = p_entry = p_ko = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [T][Hq][D], got shape %s" % (tuple(q.shape),))
        T, H, D = q.shape
        q_stride, head, one = q.stride()
        q_f32 = q.dtype is _F32
        if not q_f32 and q.dtype is not _BF16:
            raise TypeError("q must be bfloat16 or float32, got %s" % q.dtype)
        if T and (one != 1 or (H > 1 and head != D)):
            raise ValueError("q must have contiguous heads, got shape %s strides %s"
                             % (tuple(q.shape), q.stride()))
        if T <= 1:
            q_stride = H * D
        if q_out is None:
            q_out = torch.empty((T, H, D), dtype=_BF16, device=q.device)
        elif q_out.shape != q.shape:
            raise ValueError("q_out must be shaped as q")
        if pos is None:
            raise ValueError("q needs pos")
        p_q, p_qo = _at(q, "q", index), _vec(q_out, "q_out", _BF16, T * H * D, index)
        p_pos = _vec(pos, "pos", _I32, T, index)
        if q_weight is not None:
            p_qw = _vec(q_weight, "q_weight", _F32, D, index)
    if kv is not None:
        if kv.dim() != 2:
            raise ValueError("kv must be [E][D], got shape %s" % (tuple(kv.shape),))
        E, channels = kv.shape
        kv_stride, one = kv.stride()
        kv_f32 = kv.dtype is _F32
        if not kv_f32 and kv.dtype is not _BF16:
            raise TypeError("kv must be bfloat16 or float32, got %s" % kv.dtype)
        if E and one != 1:
            raise ValueError("kv must have contiguous rows, got strides %s" % (kv.stride(),))
        if q is not None and channels != D:
            raise ValueError("q and kv must have as many channels, got %d and %d" % (D, channels))
        D = channels
        if E <= 1:
            kv_stride = D
        if pages is None or kv_pos is None or seq is None or entry is None:
            raise ValueError("kv needs kv_pos, pages, seq and entry")
        if pages.index != index:
            raise ValueError("pages must be on cuda:%d, got %s" % (index, pages.device))
        p_kv = _at(kv, "kv", index)
        p_kp = _vec(kv_pos, "kv_pos", _I32, E, index)
        p_seq = _vec(seq, "seq", _I32, E, index)
        p_entry = _vec(entry, "entry", _I32, E, index)
        if kv_weight is not None:
            p_kw = _vec(kv_weight, "kv_weight", _F32, D, index)
        if kv_out is not None:
            if kv_out.shape != kv.shape:
                raise ValueError("kv_out must be shaped as kv")
            p_ko = _vec(kv_out, "kv_out", _BF16, E * D, index)
    if index < 0:
        raise ValueError("expected CUDA tensors")
    args = NormRopeArgs.from_buffer_copy(_ROPE_PACK.pack(
        D, 2 * R2, rot_begin, bool(interleaved), bool(inverse), rot_scale, eps, p_turns, T, H,
        bool(q_norm), q_f32, p_q, q_stride, p_pos, p_qw, p_qo, E, bool(kv_norm), kv_f32, p_kv,
        kv_stride, p_kp, p_kw, p_seq, p_entry, p_ko))
    _call("csa2_qk_norm_rope", index, ctypes.byref(args), pages.ref if pages is not None else None)
    return q_out, kv_out


def csa2_paged_attn(q: torch.Tensor, pages: Fp4Pages, softmax_scale: float,
                    seq: Optional[torch.Tensor] = None, nvalid: Optional[torch.Tensor] = None,
                    topk_idx: Optional[torch.Tensor] = None, want_lse: bool = True,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None):
    """q bf16 [B][Tq][Hq][512] over slots seq int32 [B] (None: slot b) of a paged
    cache: all of the first nvalid int32 [B][Tq] entries (None: the slot's length),
    or those listed in topk_idx int32 [B][Tq][K] -> (out bf16, lse float32 or None)."""
    if q.dim() != 4:
        raise ValueError("q must be [B][Tq][Hq][D], got shape %s" % (tuple(q.shape),))
    B, Tq, H, D = q.shape
    index, device = pages.index, pages.device
    if D != pages.D:
        raise ValueError("q has %d channels, the pages %d" % (D, pages.D))
    p_q = _vec(q, "q", _BF16, B * Tq * H * D, index)
    p_seq = None if seq is None else _vec(seq, "seq", _I32, B, index)
    p_nv = None if nvalid is None else _vec(nvalid, "nvalid", _I32, B * Tq, index)
    K, p_ids = 0, None
    if topk_idx is not None:
        if topk_idx.dim() != 3 or topk_idx.shape[2] == 0:
            raise ValueError("topk_idx must be [B][Tq][K] with K >= 1, got shape %s"
                             % (tuple(topk_idx.shape),))
        K = topk_idx.shape[2]
        p_ids = _vec(topk_idx, "topk_idx", _I32, B * Tq * K, index)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape:
        raise ValueError("out must be shaped as q")
    p_lse = None
    if want_lse:
        if lse is None:
            lse = torch.empty((B, Tq, H), dtype=_F32, device=device)
        elif lse.shape != q.shape[:3]:
            raise ValueError("lse must be [B][Tq][Hq]")
        p_lse = _vec(lse, "lse", _F32, B * Tq * H, index)
    ws, p, size = _scratch(workspace,
                           pages.workspace_bytes("csa2_paged_attn", B, Tq, H, K), device)
    _call("csa2_paged_attn", index, p_q, pages.ref, p_seq, p_nv, p_ids, B, Tq, H, K,
          softmax_scale, _vec(out, "out", _BF16, B * Tq * H * D, index), p_lse, p, size)
    return out, (lse if want_lse else None)
