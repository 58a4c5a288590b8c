"""Python binding of the C-ABI library (libsparstar.so): argument marshalling only.

Every step of the path (pooling, scoring, Top-K, attention) runs in the library's CUDA
kernels. Torch is used to allocate device memory and to name the current stream. The
binding raises if the library is missing: there is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

from . import _build

BLOCK = 128
BUDGET_LITERAL = 0
BUDGET_CANDIDATES = 1

OK = 0
ERR_ARG = 1
ERR_UNSUPPORTED = 2
ERR_WORKSPACE = 3
ERR_CUDA = 4
ERR_DEVICE_TIMEOUT = 5
ERR_DEVICE_BOUNDS = 6

# Every function the header declares, with (restype, argtypes).
_c = ctypes
_SIGNATURES = {}


class Segments(ctypes.Structure):
    _fields_ = [("n_text", ctypes.c_int64), ("n_ctx", ctypes.c_int64), ("n_cur", ctypes.c_int64)]


class Grid(ctypes.Structure):
    _fields_ = [("frames", ctypes.c_int64), ("height", ctypes.c_int64), ("width", ctypes.c_int64)]


class Plan(ctypes.Structure):
    _fields_ = [("nqb", ctypes.c_int64), ("nkb", ctypes.c_int64), ("n_forced", ctypes.c_int64),
                ("n_cand", ctypes.c_int64), ("k_total", ctypes.c_int32), ("k_topk", ctypes.c_int32)]

    def as_dict(self):
        return {f: int(getattr(self, f)) for f, _ in self._fields_}


_SIGNATURES.update({
    "sparstar_abi_version": (_c.c_int, []),
    "sparstar_strerror": (_c.c_char_p, [_c.c_int]),
    "sparstar_make_plan": (_c.c_int, [_c.c_int64, Segments, _c.c_int, _c.c_double, _c.c_int, _c.POINTER(Plan)]),
    "sparstar_workspace_size": (_c.c_int, [_c.c_int, _c.c_int64, Segments, _c.c_int, _c.POINTER(_c.c_size_t)]),
    "sparstar_select": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, Segments, _c.c_int, _c.c_int,
                                   _c.c_double, _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_void_p,
                                   _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "sparstar_attn": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int,
                                 _c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_float, _c.c_void_p, _c.c_void_p,
                                 _c.c_void_p]),
    "sparstar_forward": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, Segments, _c.c_int,
                                    _c.c_int, _c.c_double, _c.c_int, _c.c_float, _c.c_void_p, _c.c_void_p,
                                    _c.c_int32, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "sparstar_device_status": (_c.c_int, [_c.c_void_p, _c.c_int]),
    "sparstar_selftest_wait_timeout": (_c.c_int, [_c.c_void_p]),
    "sparstar_make_plan_ex": (_c.c_int, [_c.c_int64, Segments, _c.c_int, _c.c_double, _c.c_int, _c.c_int,
                                         _c.POINTER(Plan)]),
    "sparstar_workspace_size_ex": (_c.c_int, [_c.c_int, _c.c_int64, Segments, _c.c_int, _c.c_int,
                                              _c.POINTER(_c.c_size_t)]),
    "sparstar_select_ex": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, Segments, _c.c_int, _c.c_int,
                                      _c.c_double, _c.c_int, _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_int32,
                                      _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "sparstar_attn_ex": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int,
                                    _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_float, _c.c_void_p,
                                    _c.c_void_p, _c.c_void_p]),
    "sparstar_forward_ex": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, Segments,
                                       _c.c_int, _c.c_int, _c.c_double, _c.c_int, _c.c_int, _c.c_float, _c.c_void_p,
                                       _c.c_void_p, _c.c_int32, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t,
                                       _c.c_void_p]),
    "sparstar_select_noalloc": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, Segments, _c.c_int,
                                           _c.c_int, _c.c_double, _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_int32,
                                           _c.c_void_p]),
})
_SIGNATURES.update({
    "sparstar_retained_mass": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_void_p, _c.c_void_p,
                                          _c.c_void_p]),
    "sparstar_token_bound_workspace_size": (_c.c_int, [_c.c_int, _c.c_int64, _c.POINTER(_c.c_size_t)]),
    "sparstar_token_bound": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int,
                                        _c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_void_p, _c.c_float, _c.c_void_p,
                                        _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "sparstar_topk": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_int, _c.c_int, _c.c_int, _c.c_void_p, _c.c_void_p,
                                 _c.c_int32, _c.c_void_p]),
    "sparstar_read_probe": (_c.c_int, [_c.c_void_p, _c.c_size_t, _c.c_void_p, _c.c_void_p]),
    "sparstar_map_scores": (_c.c_int, [_c.c_void_p, _c.c_int, Segments, Grid, Segments, Grid, _c.c_void_p,
                                       _c.c_void_p]),
})


class View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("seq_stride", ctypes.c_int64)]


BF16 = 0
FP32 = 1
_X_DTYPES = {torch.bfloat16: BF16, torch.float32: FP32}
_SIGNATURES.update({
    "sparstar_qk_norm_rope": (_c.c_int, [View, View, View, _c.c_int, _c.c_int64, _c.c_int, _c.c_int, _c.c_int,
                                         _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_float, _c.c_int,
                                         View, View, View, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_void_p]),
    "sparstar_qk_norm_rope_bwd_workspace_size": (_c.c_int, [_c.c_int, _c.POINTER(_c.c_size_t)]),
    "sparstar_qk_norm_rope_bwd": (_c.c_int, [View, View, View, View, View, _c.c_int, _c.c_int64, _c.c_int, _c.c_int,
                                             _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_float,
                                             _c.c_int, _c.c_int64, View, View, View, _c.c_void_p, _c.c_void_p,
                                             _c.c_void_p, _c.c_size_t, _c.c_void_p]),
})
_SIGNATURES.update({
    "sparstar_attn_bwd_workspace_size": (_c.c_int, [_c.c_int, _c.c_int64, _c.c_int64, _c.c_int, _c.c_int, _c.c_int32,
                                                    _c.POINTER(_c.c_size_t)]),
    "sparstar_attn_bwd": (_c.c_int, [_c.c_void_p] * 6 + [_c.c_int, _c.c_int64, _c.c_int64, _c.c_int, _c.c_int,
                                                         _c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_float, _c.c_void_p,
                                                         _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t,
                                                         _c.c_void_p]),
})
_TOKEN_SIZES = [_c.c_int, _c.c_int, _c.c_int, _c.c_int64, _c.c_int]
_SIGNATURES.update({
    "sparstar_block_means": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int, _c.c_int64, _c.c_int, _c.c_int,
                                        _c.c_void_p, _c.c_void_p]),
    "sparstar_token_select": (_c.c_int, [_c.c_void_p] * 3 + _TOKEN_SIZES + [_c.c_int] * 3 + [_c.c_void_p] * 3),
    "sparstar_token_attn": (_c.c_int, [_c.c_void_p] * 4 + _TOKEN_SIZES + [_c.c_void_p, _c.c_void_p, _c.c_int,
                                                                         _c.c_float, _c.c_void_p, _c.c_void_p,
                                                                         _c.c_void_p]),
    "sparstar_token_forward": (_c.c_int, [_c.c_void_p] * 5 + _TOKEN_SIZES + [_c.c_int] * 3 + [_c.c_float]
                               + [_c.c_void_p] * 5),
})
NOALLOC_SCRATCH_BYTES = 128 << 20

_LIB: Optional[ctypes.CDLL] = None


class SparstarError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} (code {code})")


def lib_path() -> str:
    return _build.LIB_PATH


def load() -> ctypes.CDLL:
    """Load libsparstar.so from the package directory (raises if it was not built)."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                               "(there is no CPU fallback)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def strerror(code: int) -> str:
    return load().sparstar_strerror(int(code)).decode()


def _check(code: int, where: str):
    if code != OK:
        raise SparstarError(code, where)


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) or None


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else int(t.data_ptr()) or None


def make_plan(n_q: int, n_text: int, n_ctx: int, n_cur: int, clip: int, density: float,
              budget_mode: int = BUDGET_LITERAL, block: int = BLOCK) -> Plan:
    plan = Plan()
    _check(load().sparstar_make_plan_ex(int(n_q), Segments(n_text, n_ctx, n_cur), int(clip), float(density),
                                        int(budget_mode), int(block), ctypes.byref(plan)), "sparstar_make_plan_ex")
    return plan


def workspace_size(heads: int, n_q: int, n_text: int, n_ctx: int, n_cur: int, head_dim: int,
                   block: int = BLOCK) -> int:
    out = ctypes.c_size_t()
    _check(load().sparstar_workspace_size_ex(int(heads), int(n_q), Segments(n_text, n_ctx, n_cur), int(head_dim),
                                             int(block), ctypes.byref(out)), "sparstar_workspace_size_ex")
    return int(out.value)


def _check_qkv(*ts):
    for t in ts:
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 3:
            raise ValueError("q/k/v must be contiguous bf16 CUDA tensors of shape [H, N, d]")


class Workspace:
    """Reusable device workspace sized for one shape (allocated once by torch)."""

    def __init__(self, heads, n_q, n_text, n_ctx, n_cur, head_dim, device, block: int = 128):
        nbytes = workspace_size(heads, n_q, n_text, n_ctx, n_cur, head_dim, block)
        self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        self.nbytes = nbytes


def select(q: torch.Tensor, k: torch.Tensor, n_text: int, n_ctx: int, n_cur: int, clip: int, density: float,
           budget_mode: int = BUDGET_LITERAL, want_scores: bool = False, workspace: Optional[Workspace] = None,
           idx: Optional[torch.Tensor] = None, cnt: Optional[torch.Tensor] = None, stream=None,
           block: int = BLOCK):
    """Block selection with `block`-token blocks (128, or 64). Returns (idx [H,nqb,K_total]
    int32, cnt [H,nqb] int32, scores or None)."""
    _check_qkv(q, k)
    H, n_q, d = q.shape
    plan = make_plan(n_q, n_text, n_ctx, n_cur, clip, density, budget_mode, block)
    nqb, nkb, kmax = int(plan.nqb), int(plan.nkb), max(int(plan.k_total), 1)
    if idx is None:
        idx = torch.empty(H, nqb, kmax, dtype=torch.int32, device=q.device)
    if cnt is None:
        cnt = torch.empty(H, nqb, dtype=torch.int32, device=q.device)
    scores = torch.empty(H, nqb, nkb, dtype=torch.float32, device=q.device) if want_scores else None
    if workspace is None:
        workspace = Workspace(H, n_q, n_text, n_ctx, n_cur, d, q.device, block)
    _check(load().sparstar_select_ex(_ptr(q), _ptr(k), H, n_q, Segments(n_text, n_ctx, n_cur), d, int(clip),
                                     float(density), int(budget_mode), int(block), _ptr(idx), _ptr(cnt),
                                     idx.shape[-1], _ptr(scores), _ptr(workspace.buf), workspace.nbytes,
                                     _stream_ptr(stream)), "sparstar_select_ex")
    return idx, cnt, scores


def attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, idx: torch.Tensor, cnt: torch.Tensor,
         sm_scale: float = 0.0, o: Optional[torch.Tensor] = None, want_lse: bool = True,
         lse: Optional[torch.Tensor] = None, stream=None, block: int = BLOCK) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Block-sparse attention over the kept tiles (`block`-token blocks). Returns (o bf16
    [H,Nq,d], lse fp32 [H,Nq] or None)."""
    _check_qkv(q, k, v)
    H, n_q, d = q.shape
    if idx.dtype != torch.int32 or cnt.dtype != torch.int32 or not idx.is_contiguous() or not cnt.is_contiguous():
        raise ValueError("idx/cnt must be contiguous int32")
    if o is None:
        o = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty(H, n_q, dtype=torch.float32, device=q.device)
    _check(load().sparstar_attn_ex(_ptr(q), _ptr(k), _ptr(v), H, n_q, k.shape[1], d, int(block), _ptr(idx),
                                   _ptr(cnt), idx.shape[-1], float(sm_scale), _ptr(o), _ptr(lse), _stream_ptr(stream)),
           "sparstar_attn_ex")
    return o, lse


def topk(scores: torch.Tensor, n_forced: int, k_topk: int, idx: Optional[torch.Tensor] = None,
         cnt: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Clip-aware retention + joint Top-K on given scores [..., nkb] (fp32, contiguous CUDA):
    each row keeps blocks 0..n_forced-1 and its k_topk best other columns, ascending.
    Returns (idx int32 [..., n_forced + k_topk] unless a wider idx is given, cnt int32 [...])."""
    if scores.dtype != torch.float32 or not scores.is_cuda or not scores.is_contiguous() or scores.dim() < 1:
        raise ValueError("scores must be a contiguous fp32 CUDA tensor [..., nkb]")
    lead, nkb = tuple(scores.shape[:-1]), scores.shape[-1]
    rows = scores.numel() // nkb if nkb else 0
    if idx is None:
        idx = torch.empty(*lead, n_forced + k_topk, dtype=torch.int32, device=scores.device)
    if cnt is None:
        cnt = torch.empty(*lead, dtype=torch.int32, device=scores.device)
    if idx.dtype != torch.int32 or cnt.dtype != torch.int32 or not idx.is_contiguous() or not cnt.is_contiguous():
        raise ValueError("idx/cnt must be contiguous int32")
    _check(load().sparstar_topk(_ptr(scores), rows, nkb, int(n_forced), int(k_topk), _ptr(idx), _ptr(cnt),
                                idx.shape[-1], _stream_ptr(stream)), "sparstar_topk")
    return idx, cnt


def _check_lse(*ts):
    for t in ts:
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() or t.dim() != 2:
            raise ValueError("LSEs must be contiguous fp32 CUDA tensors of shape [H, Nq]")


def retained_mass(lse_kept: torch.Tensor, lse_dense: torch.Tensor, want_tokens: bool = True, stream=None):
    """Retained dense softmax mass of a mask from the two LSEs of sparstar_attn (mask / all
    blocks). Returns (R fp32 [H,Nq] or None, per-query-block mean fp32 [H,nqb])."""
    _check_lse(lse_kept, lse_dense)
    H, n_q = lse_kept.shape
    nqb = -(-n_q // 128)
    r = torch.empty(H, n_q, dtype=torch.float32, device=lse_kept.device) if want_tokens else None
    e = torch.empty(H, nqb, dtype=torch.float32, device=lse_kept.device)
    _check(load().sparstar_retained_mass(_ptr(lse_kept), _ptr(lse_dense), H, n_q, _ptr(r), _ptr(e),
                                         _stream_ptr(stream)), "sparstar_retained_mass")
    return r, e


def token_bound(q: torch.Tensor, k: torch.Tensor, idx: torch.Tensor, cnt: torch.Tensor, lse_dense: torch.Tensor,
                sm_scale: float = 0.0, want_tokens: bool = True, stream=None):
    """Token-wise upper bound on the retained mass with each row's kept-token budget.
    Returns (U fp32 [H,Nq] or None, per-query-block mean fp32 [H,nqb])."""
    _check_qkv(q, k)
    _check_lse(lse_dense)
    H, n_q, d = q.shape
    if idx.dtype != torch.int32 or cnt.dtype != torch.int32 or not idx.is_contiguous() or not cnt.is_contiguous():
        raise ValueError("idx/cnt must be contiguous int32")
    nqb = -(-n_q // 128)
    nbytes = ctypes.c_size_t()
    _check(load().sparstar_token_bound_workspace_size(H, n_q, ctypes.byref(nbytes)), "sparstar_token_bound_workspace_size")
    ws = torch.empty(max(int(nbytes.value), 256), dtype=torch.uint8, device=q.device)
    u = torch.empty(H, n_q, dtype=torch.float32, device=q.device) if want_tokens else None
    ub = torch.empty(H, nqb, dtype=torch.float32, device=q.device)
    _check(load().sparstar_token_bound(_ptr(q), _ptr(k), H, n_q, k.shape[1], d, _ptr(idx), _ptr(cnt), idx.shape[-1],
                                       _ptr(lse_dense), float(sm_scale), _ptr(u), _ptr(ub), _ptr(ws), int(nbytes.value),
                                       _stream_ptr(stream)), "sparstar_token_bound")
    return u, ub


def forward(q, k, v, n_text, n_ctx, n_cur, clip, density, budget_mode=BUDGET_LITERAL, sm_scale=0.0,
            workspace: Optional[Workspace] = None, idx=None, cnt=None, o=None, lse=None, want_lse=True,
            stream=None, block: int = BLOCK):
    """The whole per-scale path (selection then attention). Returns (o, lse, idx, cnt)."""
    _check_qkv(q, k, v)
    H, n_q, d = q.shape
    plan = make_plan(n_q, n_text, n_ctx, n_cur, clip, density, budget_mode, block)
    kmax = max(int(plan.k_total), 1)
    if idx is None:
        idx = torch.empty(H, int(plan.nqb), kmax, dtype=torch.int32, device=q.device)
    if cnt is None:
        cnt = torch.empty(H, int(plan.nqb), dtype=torch.int32, device=q.device)
    if o is None:
        o = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty(H, n_q, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = Workspace(H, n_q, n_text, n_ctx, n_cur, d, q.device, block)
    _check(load().sparstar_forward_ex(_ptr(q), _ptr(k), _ptr(v), H, n_q, Segments(n_text, n_ctx, n_cur), d,
                                      int(clip), float(density), int(budget_mode), int(block), float(sm_scale),
                                      _ptr(idx), _ptr(cnt), idx.shape[-1], _ptr(o), _ptr(lse), _ptr(workspace.buf),
                                      workspace.nbytes, _stream_ptr(stream)), "sparstar_forward_ex")
    return o, lse, idx, cnt


def select_noalloc(q: torch.Tensor, k: torch.Tensor, n_text: int, n_ctx: int, n_cur: int, clip: int,
                   density: float, budget_mode: int = BUDGET_LITERAL, idx: Optional[torch.Tensor] = None,
                   cnt: Optional[torch.Tensor] = None, stream=None):
    """Block selection without any device allocation inside the library: its scratch is the
    library's fixed array (NOALLOC_SCRATCH_BYTES per device). For callers that cannot call
    cudaMalloc; they pass idx and cnt buffers they already own. Calls that overlap on the
    GPU share that array and race. Returns (idx, cnt)."""
    _check_qkv(q, k)
    H, n_q, d = q.shape
    plan = make_plan(n_q, n_text, n_ctx, n_cur, clip, density, budget_mode)
    if idx is None:
        idx = torch.empty(H, int(plan.nqb), max(int(plan.k_total), 1), dtype=torch.int32, device=q.device)
    if cnt is None:
        cnt = torch.empty(H, int(plan.nqb), dtype=torch.int32, device=q.device)
    _check(load().sparstar_select_noalloc(_ptr(q), _ptr(k), H, n_q, Segments(n_text, n_ctx, n_cur), d, int(clip),
                                          float(density), int(budget_mode), _ptr(idx), _ptr(cnt), idx.shape[-1],
                                          _stream_ptr(stream)), "sparstar_select_noalloc")
    return idx, cnt


def map_scores(scores_prev: torch.Tensor, seg_prev, grid_prev, seg_now, grid_now, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Block scores of a previous scale of the clip carried to the current scale through the
    nearest-raster-position block map (seg_* = (n_text, n_ctx, n_cur), grid_* = (frames, height,
    width) of the current tokens). Returns fp32 [H, nqb_now, nkb_now]."""
    if scores_prev.dtype != torch.float32 or not scores_prev.is_cuda or not scores_prev.is_contiguous() \
            or scores_prev.dim() != 3:
        raise ValueError("scores_prev must be a contiguous fp32 CUDA tensor [H, nqb, nkb]")
    H = scores_prev.shape[0]
    n_prefix = (seg_now[0] + seg_now[1]) // BLOCK
    nqb_now = -(-seg_now[2] // BLOCK)
    if out is None:
        out = torch.empty(H, nqb_now, n_prefix + nqb_now, dtype=torch.float32, device=scores_prev.device)
    _check(load().sparstar_map_scores(_ptr(scores_prev), H, Segments(*seg_prev), Grid(*grid_prev), Segments(*seg_now),
                                      Grid(*grid_now), _ptr(out), _stream_ptr(stream)), "sparstar_map_scores")
    return out


def read_probe(buf: torch.Tensor, sink: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Measurement aid: one streaming read of `buf` (a contiguous CUDA tensor whose size is a
    multiple of 16 bytes), XOR-folded into a 4-byte sink, which is returned."""
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous CUDA tensor")
    if sink is None:
        sink = torch.zeros(1, dtype=torch.int32, device=buf.device)
    _check(load().sparstar_read_probe(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink), _stream_ptr(stream)),
           "sparstar_read_probe")
    return sink


# ------------------------------------------------------------------ gradient of the attention

def attn_bwd_workspace_size(heads: int, n_q: int, n_kv: int, head_dim: int, kmax: int, block: int = BLOCK) -> int:
    out = ctypes.c_size_t()
    _check(load().sparstar_attn_bwd_workspace_size(int(heads), int(n_q), int(n_kv), int(head_dim), int(block),
                                                   int(kmax), ctypes.byref(out)), "sparstar_attn_bwd_workspace_size")
    return int(out.value)


class AttnBwdWorkspace:
    """Reusable device workspace of attn_bwd for one shape (kmax: width of idx). Calls that may
    overlap on the GPU need one each."""

    def __init__(self, heads, n_q, n_kv, head_dim, kmax, device, block: int = BLOCK):
        nbytes = attn_bwd_workspace_size(heads, n_q, n_kv, head_dim, kmax, block)
        self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        self.nbytes = nbytes


def attn_bwd(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
             idx: torch.Tensor, cnt: torch.Tensor, sm_scale: float = 0.0, dq: Optional[torch.Tensor] = None,
             dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
             workspace: Optional[AttnBwdWorkspace] = None, stream=None, block: int = BLOCK):
    """Gradient of attn over the same kept lists. do is the gradient of its output o; q, k, v, idx,
    cnt, sm_scale and block are its arguments, o and lse its results. Returns (dq, dk, dv), bf16,
    every element written. The same inputs give the same bits."""
    _check_qkv(do, q, k, v, o)
    H, n_q, d = q.shape
    n_kv = k.shape[1]
    nqb = -(-n_q // block) if block in (64, 128) else 0
    if do.shape != q.shape or o.shape != q.shape or k.shape != (H, n_kv, d) or v.shape != k.shape:
        raise ValueError("do and o must have q's shape [H, Nq, d], v k's shape [H, Nkv, d]")
    if lse.dtype != torch.float32 or lse.shape != (H, n_q) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [H, Nq]")
    if idx.dtype != torch.int32 or cnt.dtype != torch.int32 or not idx.is_contiguous() or not cnt.is_contiguous():
        raise ValueError("idx/cnt must be contiguous int32")
    if nqb and (idx.dim() != 3 or idx.shape[:2] != (H, nqb) or cnt.shape != (H, nqb)):
        raise ValueError(f"idx must be [H, {nqb}, kmax] and cnt [H, {nqb}]")
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None and (t.dtype != torch.bfloat16 or t.shape != like.shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous bf16 {list(like.shape)}")
    _check_device(q.device, do, k, v, o, lse, idx, cnt, dq, dk, dv, None if workspace is None else workspace.buf)
    kmax = max(int(idx.shape[-1]), 1)
    with _launch(q.device, stream) as st:
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        if workspace is None:
            workspace = AttnBwdWorkspace(H, n_q, n_kv, d, kmax, q.device, block)
        _check(load().sparstar_attn_bwd(_at(do), _at(q), _at(k), _at(v), _at(o), _at(lse), H, n_q, n_kv, d,
                                        int(block), _at(idx), _at(cnt), kmax, float(sm_scale), _at(dq), _at(dk),
                                        _at(dv), _at(workspace.buf), workspace.nbytes, st), "sparstar_attn_bwd")
    return dq, dk, dv


# ------------------------------------------------------------------ norm, rotation, head layout

class _launch:
    """Makes `device` and `stream` (None: the device's current stream) current, so that buffers
    allocated inside belong to the stream that uses them; gives the stream's pointer. Where they
    are current already, which is the usual call, nothing is switched."""

    __slots__ = ("device", "stream", "switched")

    def __init__(self, device: torch.device, stream):
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
        self.device, self.stream, self.switched = device, stream, None

    def __enter__(self):
        if self.stream is not None or torch.cuda.current_device() != self.device.index:
            self.switched = contextlib.ExitStack()
            self.switched.enter_context(torch.cuda.device(self.device))
            if self.stream is not None:
                self.switched.enter_context(torch.cuda.stream(self.stream))
                return self.stream.cuda_stream
        # the pointer alone: a Stream object costs as much as everything else here
        return torch._C._cuda_getCurrentRawStream(self.device.index)

    def __exit__(self, *exc):
        if self.switched is not None:
            self.switched.close()


def _check_device(device, *tensors):
    """All of `tensors` (None: left out) on one CUDA device."""
    if device.type != "cuda":
        raise ValueError("tensors must be CUDA tensors")
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"tensors are on {device} and {t.device}")


_NO_VIEW = View(None, 0, 0, 0)


def _at(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _view(name: str, t: Optional[torch.Tensor], shape, dtype, token: int, head: int, seq: int = -1) -> View:
    """The strided head vectors of t (None: none), checked: `shape` with the vectors contiguous."""
    if t is None:
        return _NO_VIEW
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {list(shape)}; got {t.dtype} {list(t.shape)}")
    st = t.stride()
    if st[-1] != 1 and t.numel():
        raise ValueError(f"{name}'s head vectors must be contiguous")
    d = shape[-1]  # stands in for the stride of a dimension of one, which addresses nothing
    return View(t.data_ptr(), st[token] if shape[token] > 1 else d, st[head] if shape[head] > 1 else d,
                0 if seq < 0 else st[seq] if shape[seq] > 1 else d)


def _norm_rope_sizes(q, k, wq, wk, cos, sin):
    """Checks of what both directions share. Returns (N, Hq, Hk, d)."""
    if q.dim() != 3 or q.dtype not in _X_DTYPES:
        raise ValueError("q must be a bf16 or fp32 CUDA tensor [N, heads, d]")
    n, hq, d = q.shape
    hk = 0
    if k is not None:
        if k.dim() != 3:
            raise ValueError("k must be [N, heads, d]")
        hk = k.shape[1]
    for name, t, shape in (("wq", wq, (d,)), ("wk", wk, (d,)), ("cos", cos, (n, d // 2)), ("sin", sin, (n, d // 2))):
        if t is not None and (t.shape != shape or t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {list(shape)}")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    return n, hq, hk, d


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                 wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None,
                 cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                 kv_rows: Optional[torch.Tensor] = None, kv_offset: int = 0, stream=None):
    """RMS norm of the queries and keys of each head, position rotation and the change to
    head-major, in one pass. q [N, Hq, d], k and v [N, Hk, d]: bf16 or fp32, any token and head
    strides (slices of one fused projection). wq, wk fp32 [d]; cos, sin fp32 [N, d/2]. Returns
    (q_out, k_out, v_out), bf16; given outputs may be strided views.

    q_out [Hq, N, d]. k_out and v_out [Hk, rows, d] receive token n at row kv_offset + n (default:
    kv_offset + N rows, those before the offset unwritten), or at row kv_rows[n] (int32 [N]). With
    kv_rows they may also be a cache [N, Hk, rows, d] that takes one token of each of N sequences.
    A negative kv_rows[n] leaves token n out; one past the rows does too and is reported by
    device_status()."""
    n, hq, hk, d = _norm_rope_sizes(q, k, wq, wk, cos, sin)
    kv_offset = int(kv_offset)
    if v is not None and k is None:
        raise ValueError("v comes with k")
    if (k_out is not None and k is None) or (v_out is not None and v is None):
        raise ValueError("k_out comes with k, and v_out with v")
    if kv_offset < 0:
        raise ValueError("kv_offset must not be negative")
    if kv_rows is not None:
        if kv_rows.dtype != torch.int32 or kv_rows.shape != (n,) or not kv_rows.is_contiguous():
            raise ValueError("kv_rows must be a contiguous int32 tensor [N]")
        if kv_offset or (k is not None and k_out is None) or (v is not None and v_out is None):
            raise ValueError("kv_rows needs k_out (and v_out) and takes no kv_offset")
    device, x_dtype, bf16 = q.device, q.dtype, torch.bfloat16
    qv, kv = _view("q", q, (n, hq, d), x_dtype, 0, 1), _view("k", k, (n, hk, d), x_dtype, 0, 1)
    vv = _view("v", v, (n, hk, d), x_dtype, 0, 1)
    _check_device(device, k, v, wq, wk, cos, sin, q_out, k_out, v_out, kv_rows)
    with _launch(device, stream) as st:
        if q_out is None:
            q_out = q.new_empty((hq, n, d), dtype=bf16)
        if k is not None and k_out is None:
            k_out = q.new_empty((hk, kv_offset + n, d), dtype=bf16)
        rows, kv_shape, dims = 0, None, (1, 0)
        if k_out is not None:
            rows, kv_shape = k_out.shape[-2], (hk, k_out.shape[-2], d)
            if kv_rows is not None and k_out.dim() == 4:
                kv_shape, dims = (n, *kv_shape), (2, 1, 0)
        if v is not None and v_out is None:
            v_out = q.new_empty((hk, kv_offset + n, d) if kv_shape is None else kv_shape, dtype=bf16)
        _check(load().sparstar_qk_norm_rope(
            qv, kv, vv, _X_DTYPES[x_dtype], n, hq, hk, d, _at(wq), _at(wk), _at(cos), _at(sin), eps, interleaved,
            _view("q_out", q_out, (hq, n, d), bf16, 1, 0), _view("k_out", k_out, kv_shape, bf16, *dims),
            _view("v_out", v_out, kv_shape, bf16, *dims), _at(kv_rows), kv_offset, rows, st), "sparstar_qk_norm_rope")
    return q_out, k_out, v_out


def qk_norm_rope_bwd(dq: torch.Tensor, dk: Optional[torch.Tensor], q: torch.Tensor, k: Optional[torch.Tensor] = None,
                     dv: Optional[torch.Tensor] = None, wq: Optional[torch.Tensor] = None,
                     wk: Optional[torch.Tensor] = None, cos: Optional[torch.Tensor] = None,
                     sin: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                     kv_offset: int = 0, dq_in: Optional[torch.Tensor] = None, dk_in: Optional[torch.Tensor] = None,
                     dv_in: Optional[torch.Tensor] = None, stream=None):
    """Gradient of qk_norm_rope (without kv_rows). dq [Hq, N, d], dk and dv [Hk, rows, d] (read at
    rows kv_offset + n): bf16, strided views allowed. q and k are the forward call's inputs.
    Returns (dq_in, dk_in, dv_in, dwq, dwk): token-major in q's type (given outputs may be slices
    of one fused gradient) and fp32 [d] sums, dwq and dwk also where the weights were left out.
    The same inputs give the same bits."""
    n, hq, hk, d = _norm_rope_sizes(q, k, wq, wk, cos, sin)
    kv_offset = int(kv_offset)
    if (dk is None) != (k is None) or (dv is not None and k is None):
        raise ValueError("dk comes with k, and dv with both")
    if (dk_in is not None and dk is None) or (dv_in is not None and dv is None):
        raise ValueError("dk_in comes with dk, and dv_in with dv")
    device, x_dtype, bf16 = q.device, q.dtype, torch.bfloat16
    views = [_view("dq", dq, (hq, n, d), bf16, 1, 0)]
    for name, t in (("dk", dk), ("dv", dv)):
        rows = t.shape[1] if t is not None and t.dim() == 3 else 0
        views.append(_view(name, t, (hk, rows, d), bf16, 1, 0))
        if t is not None and (kv_offset < 0 or kv_offset + n > rows):
            raise ValueError(f"{name} has no rows {kv_offset} to {kv_offset + n}")
    views += [_view("q", q, (n, hq, d), x_dtype, 0, 1), _view("k", k, (n, hk, d), x_dtype, 0, 1)]
    _check_device(device, dq, dk, dv, k, wq, wk, cos, sin, dq_in, dk_in, dv_in)
    with _launch(device, stream) as st:
        if dq_in is None:
            dq_in = q.new_empty((n, hq, d))
        if dk is not None and dk_in is None:
            dk_in = q.new_empty((n, hk, d))
        if dv is not None and dv_in is None:
            dv_in = q.new_empty((n, hk, d))
        dw = q.new_empty((2, d), dtype=torch.float32)
        nbytes = _norm_rope_bwd_workspace_size(d)
        ws = q.new_empty(nbytes, dtype=torch.uint8)
        at = dw.data_ptr()
        _check(load().sparstar_qk_norm_rope_bwd(
            *views, _X_DTYPES[x_dtype], n, hq, hk, d, _at(wq), _at(wk), _at(cos), _at(sin), eps, interleaved,
            kv_offset, _view("dq_in", dq_in, (n, hq, d), x_dtype, 0, 1),
            _view("dk_in", dk_in, (n, hk, d), x_dtype, 0, 1), _view("dv_in", dv_in, (n, hk, d), x_dtype, 0, 1), at,
            at + 4 * d if dk is not None else None, ws.data_ptr(), nbytes, st), "sparstar_qk_norm_rope_bwd")
    dwq, dwk = dw.unbind(0)
    return dq_in, dk_in, dv_in, dwq, dwk if dk is not None else None


@functools.lru_cache(maxsize=None)
def _norm_rope_bwd_workspace_size(head_dim: int) -> int:
    out = ctypes.c_size_t()
    _check(load().sparstar_qk_norm_rope_bwd_workspace_size(head_dim, ctypes.byref(out)),
           "sparstar_qk_norm_rope_bwd_workspace_size")
    return int(out.value)


# ------------------------------------------------------------------ one query token per sequence

def _check_cache(k, v, kv_len, means, q=None):
    """Checks of a cache and what belongs to it. Returns (B, Hk, S, d)."""
    if k.dim() != 4 or k.dtype != torch.bfloat16 or not k.is_contiguous():
        raise ValueError("a cache must be a contiguous bf16 CUDA tensor [B, Hk, S, d]")
    b, hk, s, d = k.shape
    if v is not None and (v.shape != k.shape or v.dtype != k.dtype or not v.is_contiguous()):
        raise ValueError("v must be a cache of k's shape")
    if means is not None:
        _check_means(means, b, hk, -(-s // BLOCK), d)
    _check_kv_len(kv_len, b)
    if q is not None:
        _check_token_q(q, b, hk, d)
    _check_device(k.device, k, v, kv_len, means, q)
    return b, hk, s, d


def _check_means(means, b, hk, nb, d):
    if means.dtype != torch.float32 or means.shape != (b, hk, nb, d) or not means.is_contiguous():
        raise ValueError(f"means must be contiguous fp32 {[b, hk, nb, d]}")


def _check_kv_len(kv_len, b):
    if kv_len.dtype != torch.int32 or kv_len.shape != (b,) or not kv_len.is_contiguous():
        raise ValueError("kv_len must be contiguous int32 [B]")


def _check_token_q(q, b, hk, d):
    if q.dim() != 3 or q.dtype != torch.bfloat16 or not q.is_contiguous() or q.shape[0] != b or q.shape[2] != d \
            or hk < 1 or q.shape[1] < 1 or q.shape[1] % hk:
        raise ValueError(f"q must be contiguous bf16 [{b}, Hq, {d}] with Hq a multiple of {hk}")


def _check_lists(idx, cnt, b, hk, keep):
    for name, t, shape in (("idx", idx, (b, hk, keep)), ("cnt", cnt, (b, hk))):
        if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous int32 {list(shape)}")


def _check_token_out(o, lse, q):
    if o is not None and (o.dtype != torch.bfloat16 or o.shape != q.shape or not o.is_contiguous()):
        raise ValueError("o must be contiguous bf16 of q's shape")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:2] or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous fp32 [B, Hq]")


class TokenWorkspace:
    """Reusable room of token_forward for one shape: the kept lists, through which the CTAs of a
    launch pass the choice on. The idx and cnt that a call with it returns lie in it until the next
    such call. Calls that may overlap on the GPU need one each."""

    def __init__(self, n_seq, heads_q, heads_k, capacity, head_dim, keep, device):
        self.shape = tuple(int(x) for x in (n_seq, heads_q, heads_k, capacity, head_dim, keep))
        n_seq, heads_q, heads_k, capacity, head_dim, keep = self.shape
        if n_seq < 0 or min(self.shape[1:]) < 1:
            raise ValueError(f"no call has {n_seq} sequences, {heads_q} and {heads_k} heads, {capacity} tokens, "
                             f"head_dim {head_dim} and {keep} blocks")
        self.buf = torch.empty(n_seq * heads_k * (keep + 1), dtype=torch.int32, device=device)
        at = n_seq * heads_k * keep
        self.idx, self.cnt = self.buf[:at].view(n_seq, heads_k, keep), self.buf[at:].view(n_seq, heads_k)

    def check(self, *shape):
        """Refuses a call of another shape."""
        if shape != self.shape:
            raise ValueError(f"the workspace is for (sequences, query heads, key heads, capacity, head_dim, keep) = "
                             f"{self.shape}, the call has {shape}")


def block_means(k: torch.Tensor, kv_len: torch.Tensor, means: Optional[torch.Tensor] = None, tail_only: bool = False,
                stream=None) -> torch.Tensor:
    """Means of the 128-token blocks of a cache k [B, Hk, S, d] of which sequence b holds kv_len[b]
    tokens: of every block that holds some, or (tail_only) of each sequence's last one. Writes and
    returns means, fp32 [B, Hk, ceil(S/128), d]; blocks without tokens keep what was there (zeros
    where means is not given)."""
    b, hk, s, d = _check_cache(k, None, kv_len, means)
    with _launch(k.device, stream) as st:
        if means is None:
            means = torch.zeros(b, hk, -(-s // BLOCK), d, dtype=torch.float32, device=k.device)
        _check(load().sparstar_block_means(_at(k), _at(kv_len), b, hk, s, d, int(tail_only), _at(means), st),
               "sparstar_block_means")
    return means


def token_select(q: torch.Tensor, means: torch.Tensor, kv_len: torch.Tensor, keep: int, n_sink: int = 1,
                 n_recent: int = 1, idx: Optional[torch.Tensor] = None, cnt: Optional[torch.Tensor] = None,
                 stream=None, capacity: Optional[int] = None):
    """Blocks that one query token per sequence, q [B, Hq, d], keeps: per (sequence, key head) the
    first n_sink, the last n_recent and the best others by the query heads' score against the
    block means, `keep` in all (every block where a sequence has no more). capacity is the cache's S,
    beyond which a length is clamped and reported (default: whole blocks). Returns (idx int32
    [B, Hk, keep], ascending, -1 behind the last, and cnt int32 [B, Hk])."""
    if means.dim() != 4:
        raise ValueError("means must be contiguous fp32 [B, Hk, blocks, d]")
    b, hk, nb, d = means.shape
    keep = int(keep)
    capacity = nb * BLOCK if capacity is None else int(capacity)
    if -(-capacity // BLOCK) != nb:
        raise ValueError(f"a capacity of {capacity} tokens does not have {nb} blocks")
    _check_means(means, b, hk, nb, d)
    _check_kv_len(kv_len, b)
    _check_token_q(q, b, hk, d)
    _check_lists(idx, cnt, b, hk, keep)
    _check_device(q.device, means, kv_len, idx, cnt)
    with _launch(q.device, stream) as st:
        idx = q.new_empty((b, hk, max(keep, 0)), dtype=torch.int32) if idx is None else idx
        cnt = q.new_empty((b, hk), dtype=torch.int32) if cnt is None else cnt
        _check(load().sparstar_token_select(_at(q), _at(means), _at(kv_len), b, q.shape[1], hk, capacity, d, keep,
                                            int(n_sink), int(n_recent), _at(idx), _at(cnt), st),
               "sparstar_token_select")
    return idx, cnt


def token_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_len: torch.Tensor, idx: torch.Tensor,
               cnt: torch.Tensor, sm_scale: float = 0.0, o: Optional[torch.Tensor] = None, want_lse: bool = True,
               lse: Optional[torch.Tensor] = None, stream=None):
    """Attention of one query token per sequence, q [B, Hq, d], over the blocks idx[..., :cnt] of the
    cache k, v [B, Hk, S, d] that holds kv_len [B] tokens. Returns (o bf16 [B, Hq, d], lse fp32
    [B, Hq] or None); with no kept token o is 0 and lse -inf."""
    b, hk, s, d = _check_cache(k, v, kv_len, None, q)
    if idx.dim() != 3:
        raise ValueError("idx must be contiguous int32 [B, Hk, keep]")
    _check_lists(idx, cnt, b, hk, idx.shape[2])
    _check_token_out(o, lse, q)
    _check_device(q.device, idx, cnt, o, lse)
    with _launch(q.device, stream) as st:
        o = torch.empty_like(q) if o is None else o
        if want_lse and lse is None:
            lse = q.new_empty((b, q.shape[1]), dtype=torch.float32)
        _check(load().sparstar_token_attn(_at(q), _at(k), _at(v), _at(kv_len), b, q.shape[1], hk, s, d, _at(idx),
                                          _at(cnt), idx.shape[2], float(sm_scale), _at(o), _at(lse), st),
               "sparstar_token_attn")
    return o, lse


def token_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_len: torch.Tensor, means: torch.Tensor,
                  keep: int, n_sink: int = 1, n_recent: int = 1, sm_scale: float = 0.0,
                  o: Optional[torch.Tensor] = None, want_lse: bool = True, lse: Optional[torch.Tensor] = None,
                  idx: Optional[torch.Tensor] = None, cnt: Optional[torch.Tensor] = None, stream=None,
                  workspace: Optional[TokenWorkspace] = None):
    """token_select and token_attn over its choice, in one launch. The lists go to idx and cnt where
    they are given, else to the workspace's, else to new ones. Returns (o, lse, idx, cnt)."""
    b, hk, s, d = _check_cache(k, v, kv_len, means, q)
    keep = int(keep)
    if workspace is not None:
        workspace.check(b, q.shape[1], hk, s, d, keep)
        idx = workspace.idx if idx is None else idx
        cnt = workspace.cnt if cnt is None else cnt
    _check_lists(idx, cnt, b, hk, keep)
    _check_token_out(o, lse, q)
    _check_device(q.device, idx, cnt, o, lse)
    with _launch(q.device, stream) as st:
        idx = q.new_empty((b, hk, max(keep, 0)), dtype=torch.int32) if idx is None else idx
        cnt = q.new_empty((b, hk), dtype=torch.int32) if cnt is None else cnt
        o = torch.empty_like(q) if o is None else o
        if want_lse and lse is None:
            lse = q.new_empty((b, q.shape[1]), dtype=torch.float32)
        _check(load().sparstar_token_forward(_at(q), _at(k), _at(v), _at(kv_len), _at(means), b, q.shape[1], hk,
                                             s, d, keep, int(n_sink), int(n_recent), float(sm_scale), _at(idx),
                                             _at(cnt), _at(o), _at(lse), st), "sparstar_token_forward")
    return o, lse, idx, cnt


def device_status(clear: bool = True, stream=None) -> int:
    """Synchronize and return the device status code (OK, ERR_DEVICE_TIMEOUT or ERR_DEVICE_BOUNDS)."""
    return int(load().sparstar_device_status(_stream_ptr(stream), 1 if clear else 0))


def selftest_wait_timeout(stream=None) -> None:
    """Enqueue the bounded-wait self-test: the next device_status() reports ERR_DEVICE_TIMEOUT."""
    _check(load().sparstar_selftest_wait_timeout(_stream_ptr(stream)), "sparstar_selftest_wait_timeout")


def exported_symbols():
    return list(_SIGNATURES)
