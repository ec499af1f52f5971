"""ctypes binding of libdhsa (the C ABI in include/dhsa.h).

Argument marshalling only: torch tensors are checked for dtype, shape,
contiguity and device, then their data pointers and the current CUDA stream
are handed to the library; the calls made once per new token are checked and
made by a compiled module (csrc/marshal.cpp). Every step of the path runs in the library's CUDA
kernels; there is no fallback. If the library is missing, loading fails
loudly (build it with `python -m long_context_prefill_dhsa_b200.build`).
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import math
import os
import re
import warnings
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdhsa.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "dhsa.h")

DHSA_OK = 0
STATUS_NAMES = {0: "DHSA_OK", 1: "DHSA_ERR_INVALID_ARG", 2: "DHSA_ERR_UNSUPPORTED", 3: "DHSA_ERR_CUDA",
                4: "DHSA_ERR_DEVICE", 5: "DHSA_ERR_WORKSPACE"}
DEVFLAG_WAIT_TIMEOUT, DEVFLAG_BAD_OFFSETS, DEVFLAG_BAD_SELECTION = 0x1, 0x2, 0x4
DEVFLAG_BAD_CACHE, DEVFLAG_BAD_TREE = 0x8, 0x10


class DHSAError(RuntimeError):
    def __init__(self, status: int, where: str, cuda_error: int = 0, flags: int = 0):
        self.status, self.where, self.cuda_error, self.flags = status, where, cuda_error, flags
        msg = f"{where}: {STATUS_NAMES.get(status, status)}"
        if cuda_error:
            msg += f" (cudaError {cuda_error})"
        if flags:
            msg += f" (device flags 0x{flags:x})"
        super().__init__(msg)


_c = ctypes
_P, _I, _F, _SZ = _c.c_void_p, _c.c_int, _c.c_float, _c.c_size_t
_SIGNATURES = {
    "dhsa_status_string": (_c.c_char_p, [_I]),
    "dhsa_last_cuda_error": (_I, []),
    "dhsa_version": (_I, []),
    "dhsa_check_device_status": (_I, [_P, _c.POINTER(_c.c_uint32)]),
    "dhsa_validate_offsets": (_I, [_P, _P, _I, _I, _I, _P]),
    "dhsa_chunk_pool": (_I, [_P, _I, _I, _I, _I, _P, _P, _I, _P, _P]),
    "dhsa_chunk_pool_qk": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P]),
    "dhsa_sel_stride": (_I, [_I, _I]),
    "dhsa_score_topk_workspace_size": (_SZ, [_I, _I, _I]),
    "dhsa_chunk_score_topk": (_I, [_P, _P, _I, _I, _I, _I, _P, _I, _P, _P, _P, _SZ, _P]),
    "dhsa_chunk_score_topk_csr": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "dhsa_budget_max_chunks": (_I, []),
    "dhsa_chunk_score_select_budget": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _I, _I, _P, _P, _P, _SZ, _P]),
    "dhsa_route_fused_workspace_size": (_SZ, [_I, _I, _I]),
    "dhsa_route_fused": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "dhsa_route_topk_csr": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _SZ,
                                 _P]),
    "dhsa_csr_nnz_upper": (_SZ, [_I, _I, _I, _I]),
    "dhsa_build_block_csr": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "dhsa_sparse_attn_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "dhsa_sparse_attn_fwd": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P, _F, _P, _P, _SZ, _P]),
    "dhsa_sparse_attn_fwd_noalloc": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P, _F, _P, _P]),
    "dhsa_sparse_attn_tiles_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "dhsa_sparse_attn_fwd_tiles": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P, _F, _I, _P, _P, _SZ,
                                        _P]),
    "dhsa_rotary_qkv": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _I, _I, _F, _P, _P, _P, _P, _P, _P,
                             _P, _P, _P, _I, _P, _P]),
    "dhsa_tree_max_drafts": (_I, []),
    "dhsa_tree_attn_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "dhsa_tree_attn": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _F, _P, _P, _P, _P, _P, _SZ, _P]),
    "dhsa_cache_evict_workspace_size": (_SZ, [_I, _I, _I]),
    "dhsa_cache_evict": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P,
                              _SZ, _P]),
    "dhsa_debug_arm_wait_timeout": (_I, [_I, _c.c_uint64]),
}

_lib: Optional[ctypes.CDLL] = None
_marshal = None


def load() -> ctypes.CDLL:
    """Load libdhsa.so (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m long_context_prefill_dhsa_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


class _ChecksInPython:
    """Stands in for the compiled checks where they are not built for this torch and Python."""

    @staticmethod
    def _leave(*args):
        return None

    rotary_qkv = tree_attn = cache_evict = _leave


def _load_marshal():
    """Load the compiled checks (csrc/marshal.cpp) of the cache's calls, which
    make them, for the library that load() has. Without a file for this very
    torch and Python the same checks run in Python, a few us a call slower."""
    global _marshal
    if _marshal is None:
        from . import build
        lib = load()
        path = build.marshal_path()
        if not os.path.exists(path):
            warnings.warn(f"{path} is missing, arguments are checked in Python: build it with "
                          "`python -m long_context_prefill_dhsa_b200.build`")
            _marshal = _ChecksInPython
            return _marshal
        spec = importlib.util.spec_from_file_location(__package__ + "._marshal", path)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.dhsa_rotary_qkv, lib.dhsa_tree_attn, lib.dhsa_tree_attn_workspace_size, lib.dhsa_cache_evict,
            lib.dhsa_cache_evict_workspace_size)))
        _marshal = m
    return _marshal


def header_functions() -> list[str]:
    """Names of the functions include/dhsa.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(dhsa_[a-z0-9_]+)\s*\(", text)))


def _check(status: int, where: str):
    if status != DHSA_OK:
        raise DHSAError(status, where, load().dhsa_last_cuda_error() if status == 3 else 0)


def _stream_ptr() -> int:
    return torch.cuda.current_stream().cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype, shape, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


# ----------------------------------------------------------------- stage calls
def check_device_status() -> int:
    flags = ctypes.c_uint32(0)
    st = load().dhsa_check_device_status(_stream_ptr(), ctypes.byref(flags))
    if st != DHSA_OK:
        raise DHSAError(st, "dhsa_check_device_status", load().dhsa_last_cuda_error() if st == 3 else 0,
                        flags.value)
    return flags.value


def debug_arm_wait_timeout(mode: int, limit_ns: int = 0):
    """Test hook of the bounded device waits (include/dhsa.h, 5): mode 1 makes
    the next attention call's first waits run out after limit_ns (the
    prefill's or that of drafted tokens), mode 2 the next fused-routing
    launch's first grid barrier; 0 disarms."""
    _check(load().dhsa_debug_arm_wait_timeout(mode, limit_ns), "dhsa_debug_arm_wait_timeout")


def validate_offsets(off: torch.Tensor, n_chunks: torch.Tensor, L: int):
    B, n1 = off.shape
    _need(off, torch.int32, None, "off")
    _need(n_chunks, torch.int32, (B,), "n_chunks")
    _check(load().dhsa_validate_offsets(_ptr(off), _ptr(n_chunks), B, n1 - 1, L, _stream_ptr()),
           "dhsa_validate_offsets")


def chunk_pool(X: torch.Tensor, off: torch.Tensor, n_chunks: torch.Tensor, out: Optional[torch.Tensor] = None):
    """Xp[b,h,c] = sum of chunk c's rows / sqrt(n_c), fp32 [B,H,Nmax,128]."""
    B, H, L, d = X.shape
    nmax = off.shape[1] - 1
    _need(X, torch.bfloat16, None, "X")
    _need(off, torch.int32, (B, nmax + 1), "off")
    _need(n_chunks, torch.int32, (B,), "n_chunks")
    if out is None:
        out = torch.empty((B, H, nmax, d), dtype=torch.float32, device=X.device)
    _need(out, torch.float32, (B, H, nmax, d), "out")
    _check(load().dhsa_chunk_pool(_ptr(X), B, H, L, d, _ptr(off), _ptr(n_chunks), nmax, _ptr(out), _stream_ptr()),
           "dhsa_chunk_pool")
    return out


def chunk_pool_qk(Q: torch.Tensor, K: torch.Tensor, off: torch.Tensor, n_chunks: torch.Tensor,
                  Qp: Optional[torch.Tensor] = None, Kp: Optional[torch.Tensor] = None):
    """Both poolings in one launch; same values as chunk_pool(Q) and chunk_pool(K)."""
    B, Hq, L, d = Q.shape
    Hkv = K.shape[1]
    nmax = off.shape[1] - 1
    _need(Q, torch.bfloat16, None, "Q")
    _need(K, torch.bfloat16, (B, Hkv, L, d), "K")
    _need(off, torch.int32, (B, nmax + 1), "off")
    _need(n_chunks, torch.int32, (B,), "n_chunks")
    if Qp is None:
        Qp = torch.empty((B, Hq, nmax, d), dtype=torch.float32, device=Q.device)
    if Kp is None:
        Kp = torch.empty((B, Hkv, nmax, d), dtype=torch.float32, device=Q.device)
    _need(Qp, torch.float32, (B, Hq, nmax, d), "Qp")
    _need(Kp, torch.float32, (B, Hkv, nmax, d), "Kp")
    _check(load().dhsa_chunk_pool_qk(_ptr(Q), _ptr(K), B, Hq, Hkv, L, d, _ptr(off), _ptr(n_chunks), nmax, _ptr(Qp),
                                     _ptr(Kp), _stream_ptr()), "dhsa_chunk_pool_qk")
    return Qp, Kp


def sel_stride(k: int, nmax: int) -> int:
    return load().dhsa_sel_stride(k, nmax)


def chunk_score_topk_csr(Qp: torch.Tensor, Kp: torch.Tensor, off: torch.Tensor, n_chunks: torch.Tensor, k: int,
                         sel: torch.Tensor, n_sel: torch.Tensor, row_ptr: torch.Tensor, col_idx: torch.Tensor,
                         cost: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Top-k selection that also writes the block CSR (include/dhsa.h, 2b):
    the results of chunk_score_topk followed by build_block_csr."""
    B, Hq, nmax, d = Qp.shape
    Hkv = Kp.shape[1]
    _need(Qp, torch.float32, None, "Qp")
    _need(Kp, torch.float32, (B, Hkv, nmax, d), "Kp")
    _need(off, torch.int32, (B, nmax + 1), "off")
    _need(n_chunks, torch.int32, (B,), "n_chunks")
    lib = load()
    stride = lib.dhsa_sel_stride(k, nmax)
    _need(sel, torch.int32, (B, Hq, nmax, stride), "sel")
    _need(n_sel, torch.int32, (B, Hq, nmax), "n_sel")
    _need(row_ptr, torch.int32, (B * Hq * nmax + 1,), "row_ptr")
    _need(col_idx, torch.int32, None, "col_idx")
    if col_idx.numel() < lib.dhsa_csr_nnz_upper(B, Hq, nmax, k):
        raise ValueError("col_idx: smaller than dhsa_csr_nnz_upper")
    if cost is not None:
        _need(cost, torch.int64, (B * Hq * nmax,), "cost")
    if workspace is None:
        workspace = torch.empty(lib.dhsa_score_topk_workspace_size(B, Hq, nmax), dtype=torch.uint8, device=Qp.device)
    _check(lib.dhsa_chunk_score_topk_csr(_ptr(Qp), _ptr(Kp), B, Hq, Hkv, nmax, _ptr(off), _ptr(n_chunks), k,
                                         _ptr(sel), _ptr(n_sel), _ptr(row_ptr), _ptr(col_idx), _ptr(cost),
                                         _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _stream_ptr()), "dhsa_chunk_score_topk_csr")
    return sel, n_sel


def chunk_score_topk(Qp: torch.Tensor, Kp: torch.Tensor, n_chunks: torch.Tensor, k: int,
                     sel: Optional[torch.Tensor] = None, n_sel: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None):
    """sel [B,Hq,Nmax,stride] (ascending, diagonal last, -1 padded) and n_sel [B,Hq,Nmax]."""
    B, Hq, nmax, d = Qp.shape
    Hkv = Kp.shape[1]
    _need(Qp, torch.float32, None, "Qp")
    _need(Kp, torch.float32, (B, Hkv, nmax, d), "Kp")
    _need(n_chunks, torch.int32, (B,), "n_chunks")
    lib = load()
    stride = lib.dhsa_sel_stride(k, nmax)
    if sel is None:
        sel = torch.empty((B, Hq, nmax, stride), dtype=torch.int32, device=Qp.device)
    if n_sel is None:
        n_sel = torch.empty((B, Hq, nmax), dtype=torch.int32, device=Qp.device)
    _need(sel, torch.int32, (B, Hq, nmax, stride), "sel")
    _need(n_sel, torch.int32, (B, Hq, nmax), "n_sel")
    ws_bytes = lib.dhsa_score_topk_workspace_size(B, Hq, nmax)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=Qp.device)
    ws_ptr = _ptr(workspace) if ws_bytes else None
    ws_len = workspace.numel() * workspace.element_size() if (ws_bytes and workspace is not None) else 0
    _check(lib.dhsa_chunk_score_topk(_ptr(Qp), _ptr(Kp), B, Hq, Hkv, nmax, _ptr(n_chunks), k, _ptr(sel),
                                     _ptr(n_sel), ws_ptr, ws_len, _stream_ptr()), "dhsa_chunk_score_topk")
    return sel, n_sel


def route_fused(Q: torch.Tensor, K: torch.Tensor, off: torch.Tensor, n_chunks: torch.Tensor, k: int,
                Qp: Optional[torch.Tensor] = None, Kp: Optional[torch.Tensor] = None,
                sel: Optional[torch.Tensor] = None, n_sel: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, row_ptr: Optional[torch.Tensor] = None,
                col_idx: Optional[torch.Tensor] = None, cost: Optional[torch.Tensor] = None):
    """Pooling of Q and K plus the top-k selection in one launch (include/dhsa.h,
    2c); the same results as chunk_pool_qk followed by chunk_score_topk. With
    row_ptr and col_idx given, the launch also writes the block CSR (2d), as
    build_block_csr would. Returns (Qp, Kp, sel, n_sel)."""
    B, Hq, L, d = Q.shape
    Hkv = K.shape[1]
    nmax = off.shape[1] - 1
    _need(Q, torch.bfloat16, None, "Q")
    _need(K, torch.bfloat16, (B, Hkv, L, d), "K")
    _need(off, torch.int32, (B, nmax + 1), "off")
    _need(n_chunks, torch.int32, (B,), "n_chunks")
    lib = load()
    stride = lib.dhsa_sel_stride(k, nmax)
    if Qp is None:
        Qp = torch.empty((B, Hq, nmax, d), dtype=torch.float32, device=Q.device)
    if Kp is None:
        Kp = torch.empty((B, Hkv, nmax, d), dtype=torch.float32, device=Q.device)
    if sel is None:
        sel = torch.empty((B, Hq, nmax, stride), dtype=torch.int32, device=Q.device)
    if n_sel is None:
        n_sel = torch.empty((B, Hq, nmax), dtype=torch.int32, device=Q.device)
    _need(Qp, torch.float32, (B, Hq, nmax, d), "Qp")
    _need(Kp, torch.float32, (B, Hkv, nmax, d), "Kp")
    _need(sel, torch.int32, (B, Hq, nmax, stride), "sel")
    _need(n_sel, torch.int32, (B, Hq, nmax), "n_sel")
    ws_bytes = lib.dhsa_route_fused_workspace_size(B, Hq, nmax)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=Q.device)
    if row_ptr is None:
        _check(lib.dhsa_route_fused(_ptr(Q), _ptr(K), B, Hq, Hkv, L, d, _ptr(off), _ptr(n_chunks), nmax, k,
                                    _ptr(Qp), _ptr(Kp), _ptr(sel), _ptr(n_sel), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream_ptr()), "dhsa_route_fused")
    else:
        _need(row_ptr, torch.int32, (B * Hq * nmax + 1,), "row_ptr")
        _need(col_idx, torch.int32, None, "col_idx")
        if col_idx.numel() < lib.dhsa_csr_nnz_upper(B, Hq, nmax, k):
            raise ValueError("col_idx: smaller than dhsa_csr_nnz_upper")
        if cost is not None:
            _need(cost, torch.int64, (B * Hq * nmax,), "cost")
        _check(lib.dhsa_route_topk_csr(_ptr(Q), _ptr(K), B, Hq, Hkv, L, d, _ptr(off), _ptr(n_chunks), nmax, k,
                                       _ptr(Qp), _ptr(Kp), _ptr(sel), _ptr(n_sel), _ptr(row_ptr), _ptr(col_idx),
                                       _ptr(cost), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _stream_ptr()), "dhsa_route_topk_csr")
    return Qp, Kp, sel, n_sel


def chunk_score_select_budget(Qp: torch.Tensor, Kp: torch.Tensor, off: torch.Tensor, n_chunks: torch.Tensor,
                              budget, recent: int, k_max: int, sel: Optional[torch.Tensor] = None,
                              n_sel: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Selection under a token budget per row (see include/dhsa.h, 2').

    `budget` is an int (every row) or an int32 CUDA tensor [B, Hq, Nmax] of
    per-row budgets. Returns sel [B,Hq,Nmax,stride(k_max)] and n_sel."""
    B, Hq, nmax, d = Qp.shape
    Hkv = Kp.shape[1]
    _need(Qp, torch.float32, None, "Qp")
    _need(Kp, torch.float32, (B, Hkv, nmax, d), "Kp")
    _need(off, torch.int32, (B, nmax + 1), "off")
    _need(n_chunks, torch.int32, (B,), "n_chunks")
    budgets = None
    if isinstance(budget, torch.Tensor):
        _need(budget, torch.int32, (B, Hq, nmax), "budget")
        budgets, budget = budget, 0
    lib = load()
    stride = lib.dhsa_sel_stride(k_max, nmax)
    if sel is None:
        sel = torch.empty((B, Hq, nmax, stride), dtype=torch.int32, device=Qp.device)
    if n_sel is None:
        n_sel = torch.empty((B, Hq, nmax), dtype=torch.int32, device=Qp.device)
    _need(sel, torch.int32, (B, Hq, nmax, stride), "sel")
    _need(n_sel, torch.int32, (B, Hq, nmax), "n_sel")
    ws_bytes = lib.dhsa_score_topk_workspace_size(B, Hq, nmax)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=Qp.device)
    ws_ptr = _ptr(workspace) if ws_bytes else None
    ws_len = workspace.numel() * workspace.element_size() if (ws_bytes and workspace is not None) else 0
    _check(lib.dhsa_chunk_score_select_budget(_ptr(Qp), _ptr(Kp), B, Hq, Hkv, nmax, _ptr(off), _ptr(n_chunks),
                                              int(budget), _ptr(budgets), recent, k_max, _ptr(sel), _ptr(n_sel),
                                              ws_ptr, ws_len, _stream_ptr()), "dhsa_chunk_score_select_budget")
    return sel, n_sel


def build_block_csr(sel: torch.Tensor, n_sel: torch.Tensor, k: int, off: torch.Tensor, n_chunks: torch.Tensor,
                    row_ptr=None, col_idx=None, cost=None, want_cost: bool = True):
    B, Hq, nmax, stride = sel.shape
    lib = load()
    _need(sel, torch.int32, None, "sel")
    _need(n_sel, torch.int32, (B, Hq, nmax), "n_sel")
    if row_ptr is None:
        row_ptr = torch.empty(B * Hq * nmax + 1, dtype=torch.int32, device=sel.device)
    if col_idx is None:
        col_idx = torch.empty(lib.dhsa_csr_nnz_upper(B, Hq, nmax, k), dtype=torch.int32, device=sel.device)
    if cost is None and want_cost:
        cost = torch.empty(B * Hq * nmax, dtype=torch.int64, device=sel.device)
    _check(lib.dhsa_build_block_csr(_ptr(sel), _ptr(n_sel), B, Hq, nmax, k, _ptr(off), _ptr(n_chunks),
                                    _ptr(row_ptr), _ptr(col_idx), _ptr(cost), _stream_ptr()),
           "dhsa_build_block_csr")
    return row_ptr, col_idx, cost


def sparse_attn_fwd(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, off: torch.Tensor, n_chunks: torch.Tensor,
                    row_ptr: torch.Tensor, col_idx: torch.Tensor, cost: Optional[torch.Tensor] = None,
                    softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, short_tiles: int = 0):
    """Attention over the kept chunk pairs. short_tiles != 0 calls the
    tile-policy entry (include/dhsa.h, 4c): 1 sends chunk tails of at most 64
    rows, 2 every row, to the 64-row kernel."""
    B, Hq, L, d = Q.shape
    Hkv = K.shape[1]
    nmax = off.shape[1] - 1
    _need(Q, torch.bfloat16, None, "Q")
    _need(K, torch.bfloat16, (B, Hkv, L, d), "K")
    _need(V, torch.bfloat16, (B, Hkv, L, d), "V")
    lib = load()
    if out is None:
        out = torch.empty_like(Q)
    _need(out, torch.bfloat16, (B, Hq, L, d), "out")
    ws_bytes = lib.dhsa_sparse_attn_tiles_workspace_size(B, Hq, L, nmax, short_tiles)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=Q.device)
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    if short_tiles == 0:
        _check(lib.dhsa_sparse_attn_fwd(_ptr(Q), _ptr(K), _ptr(V), B, Hq, Hkv, L, d, _ptr(off), _ptr(n_chunks),
                                        nmax, _ptr(row_ptr), _ptr(col_idx), _ptr(cost), scale, _ptr(out),
                                        _ptr(workspace), workspace.numel(), _stream_ptr()), "dhsa_sparse_attn_fwd")
    else:
        _check(lib.dhsa_sparse_attn_fwd_tiles(_ptr(Q), _ptr(K), _ptr(V), B, Hq, Hkv, L, d, _ptr(off),
                                              _ptr(n_chunks), nmax, _ptr(row_ptr), _ptr(col_idx), scale,
                                              int(short_tiles), _ptr(out), _ptr(workspace), workspace.numel(),
                                              _stream_ptr()), "dhsa_sparse_attn_fwd_tiles")
    return out


def sparse_attn_fwd_noalloc(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, off: torch.Tensor,
                            n_chunks: torch.Tensor, row_ptr: torch.Tensor, col_idx: torch.Tensor,
                            softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None):
    """sparse_attn_fwd with the library's static scratch instead of a caller
    workspace (for callers that cannot allocate; see include/dhsa.h, 4b).
    `out` should be preallocated by such callers."""
    B, Hq, L, d = Q.shape
    Hkv = K.shape[1]
    nmax = off.shape[1] - 1
    _need(Q, torch.bfloat16, None, "Q")
    _need(K, torch.bfloat16, (B, Hkv, L, d), "K")
    _need(V, torch.bfloat16, (B, Hkv, L, d), "V")
    if out is None:
        out = torch.empty_like(Q)
    _need(out, torch.bfloat16, (B, Hq, L, d), "out")
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    _check(load().dhsa_sparse_attn_fwd_noalloc(_ptr(Q), _ptr(K), _ptr(V), B, Hq, Hkv, L, d, _ptr(off),
                                               _ptr(n_chunks), nmax, _ptr(row_ptr), _ptr(col_idx), scale,
                                               _ptr(out), _stream_ptr()), "dhsa_sparse_attn_fwd_noalloc")
    return out


# ----------------------------------------------------------------- rotary positions and the cache
# These calls are made once per new token and layer, so a compiled module checks
# their arguments and makes them (csrc/marshal.cpp; append of one token: 11.7 ->
# 3.9 us of the host a call, an eviction 14.4 -> 4.9). What it does not take as it is comes here: another current
# device, numbers of other types, and the reasons of a refusal.
_raw_stream = torch._C._cuda_getCurrentRawStream     # current stream of a device, as an address
_Strides = ctypes.c_int64 * 3


def _on(t: Optional[torch.Tensor], dtype, shape, name: str, device: int):
    """A dense tensor of the call, on the call's device; returns its pointer (None for None)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, dtype, shape, name)
    raise ValueError(f"{name}: on {t.device}, expected cuda:{device}")


def _rows(t: Optional[torch.Tensor], shape, name: str, device: int):
    """A [B, H, rows, 128] bf16 tensor with contiguous rows and any strides:
    returns its pointer and its strides for the library (None when dense)."""
    if t is None:
        return None, None
    try:
        if t.dtype is torch.bfloat16 and t.shape == shape and t.get_device() == device:
            if t.is_contiguous():
                return t.data_ptr(), None
            if t.stride(3) != 1:
                raise ValueError(f"{name}: the 128 elements of a row must be contiguous")
            return t.data_ptr(), _Strides(*t.stride()[:3])
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name}: dtype {t.dtype}, expected torch.bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{device}")
    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _call_device(t: torch.Tensor, name: str) -> int:
    """Device number of the call's first tensor, a CUDA tensor of four dimensions."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise TypeError(f"{name}: expected a tensor of four dimensions")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: dtype {t.dtype}, expected torch.bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    return t.get_device()


@functools.lru_cache(maxsize=256)
def _tree_workspace(B: int, Hq: int, Hkv: int, T: int, cap: int, want_weight: bool) -> int:
    return load().dhsa_tree_attn_workspace_size(B, Hq, Hkv, T, cap, want_weight)


@functools.lru_cache(maxsize=256)
def _evict_workspace(B: int, Hkv: int, cap: int) -> int:
    return load().dhsa_cache_evict_workspace_size(B, Hkv, cap)


def _int32(x) -> int:
    """A count as the library takes it: beyond 32 bits the nearest int (ctypes
    would take it modulo 2^32, and "all" would become none)."""
    return max(-0x80000000, min(int(x), 0x7fffffff))


def _workspace(t: Optional[torch.Tensor], size: int, device: int):
    """Pointer and bytes of the caller's workspace, or of a new one (kept by the returned tensor)."""
    if t is None:
        t = torch.empty(size, dtype=torch.uint8, device=device)
        return t, t.data_ptr(), size
    _need(t, t.dtype, None, "workspace")
    if t.get_device() != device:
        raise ValueError(f"workspace: on {t.device}, expected cuda:{device}")
    return t, t.data_ptr(), t.numel() * t.element_size()


def rotary_qkv(Q: Optional[torch.Tensor], K: Optional[torch.Tensor], inv_freq: torch.Tensor,
               V: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
               start: Optional[torch.Tensor] = None, n_new: Optional[torch.Tensor] = None,
               slots: Optional[torch.Tensor] = None, interleaved: bool = False, transpose: bool = False,
               factor: float = 1.0, Q_out: Optional[torch.Tensor] = None, K_out: Optional[torch.Tensor] = None,
               V_out: Optional[torch.Tensor] = None, pos_out: Optional[torch.Tensor] = None):
    """Rotary positions of Q and K (include/dhsa.h, 6), and K, V (copied) and
    the positions written into a cache.

    Q [B,Hq,T,128], K and V [B,Hkv,T,128] may be views (e.g. of a
    [B,T,H,128] projection); any of them may be None. inv_freq: float64
    [rotary_dim/2]. positions int32 [B,T], or start int32 [B] (start + t), or
    neither (t). K_out, V_out [B,Hkv,cap,128] receive row t at slots[b] + t
    (slots None: t); missing outputs are allocated with T rows. Rows
    t >= n_new[b] are left alone. transpose=True applies the transposed
    rotation (its gradient). Returns (Q_out, K_out, V_out)."""
    done = (_marshal or _load_marshal()).rotary_qkv(Q, K, inv_freq, V, positions, start, n_new, slots, interleaved,
                                                    transpose, factor, Q_out, K_out, V_out, pos_out)
    if done is not None:
        if type(done) is int:
            _check(done, "dhsa_rotary_qkv")
        return done
    ref = Q if Q is not None else K if K is not None else V
    if ref is None:
        raise ValueError("rotary_qkv: Q, K and V are all None")
    device = _call_device(ref, "Q" if Q is not None else "K" if K is not None else "V")
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return rotary_qkv(Q, K, inv_freq, V, positions, start, n_new, slots, interleaved, transpose, factor,
                              Q_out, K_out, V_out, pos_out)
    for t, name in ((K, "K"), (V, "V"), (K_out, "K_out"), (V_out, "V_out")):
        if t is not None:
            _call_device(t, name)
    B, _, T, d = ref.shape
    Hq = Q.shape[1] if Q is not None else 1
    kv = K if K is not None else V
    Hkv = kv.shape[1] if kv is not None else 1
    q, qs = _rows(Q, (B, Hq, T, d), "Q", device)
    k, ks = _rows(K, (B, Hkv, T, d), "K", device)
    v, vs = _rows(V, (B, Hkv, T, d), "V", device)
    if (Q is None and Q_out is not None) or (K is None and K_out is not None) or (V is None and V_out is not None):
        raise ValueError("rotary_qkv: an output is given without its input")
    if Q is not None and Q_out is None:
        Q_out = torch.empty((B, Hq, T, d), dtype=torch.bfloat16, device=device)
    cap = K_out.shape[2] if K_out is not None else V_out.shape[2] if V_out is not None else T
    if K is not None and K_out is None:
        K_out = torch.empty((B, Hkv, cap, d), dtype=torch.bfloat16, device=device)
    if V is not None and V_out is None:
        V_out = torch.empty((B, Hkv, cap, d), dtype=torch.bfloat16, device=device)
    qo = _on(Q_out, torch.bfloat16, (B, Hq, T, d), "Q_out", device)
    ko, kos = _rows(K_out, (B, Hkv, cap, d), "K_out", device)
    vo, vos = _rows(V_out, (B, Hkv, cap, d), "V_out", device)
    if not isinstance(inv_freq, torch.Tensor):
        raise TypeError("inv_freq: expected a torch.Tensor")
    if positions is not None and start is not None:
        raise ValueError("rotary_qkv: positions and start exclude each other")
    _check(load().dhsa_rotary_qkv(
        q, qs, k, ks, v, vs, B, Hq, Hkv, T, d, _on(inv_freq, torch.float64, (inv_freq.numel(),), "inv_freq", device),
        2 * inv_freq.numel(), bool(interleaved), bool(transpose), factor,
        _on(positions, torch.int32, (B, T), "positions", device), _on(start, torch.int32, (B,), "start", device),
        _on(n_new, torch.int32, (B,), "n_new", device), qo, ko, kos, vo, vos,
        _on(slots, torch.int32, (B,), "slots", device), cap,
        _on(pos_out, torch.int32, (B, Hkv, cap), "pos_out", device), _raw_stream(device)), "dhsa_rotary_qkv")
    return Q_out, K_out, V_out


def tree_max_drafts() -> int:
    return load().dhsa_tree_max_drafts()


def tree_attn(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, lengths: torch.Tensor,
              parents: Optional[torch.Tensor] = None, n_draft: Optional[torch.Tensor] = None,
              softmax_scale: Optional[float] = None, weight: Optional[torch.Tensor] = None,
              weight_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Attention of each sequence's drafted tokens over a cache (include/dhsa.h, 7).

    Q [B,Hq,T,128] dense, T <= 64; caches K, V [B,Hkv,cap,128] (views with
    contiguous rows will do); lengths int32 [B] cached slots, the drafted
    tokens' K and V in the slots after them. parents int32 [B,T] is the tree
    (None: a chain; T = 1 is plain decoding). With `weight` (fp32 [B,Hkv,cap])
    each slot's attention weight is added to it, into weight_out (None: in
    place). Returns out (bf16, like Q)."""
    done = (_marshal or _load_marshal()).tree_attn(Q, K, V, lengths, parents, n_draft, softmax_scale, weight,
                                                   weight_out, out, lse, workspace)
    if done is not None:
        if type(done) is int:
            _check(done, "dhsa_tree_attn")
        return done
    device = _call_device(Q, "Q")
    _call_device(K, "K")
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return tree_attn(Q, K, V, lengths, parents, n_draft, softmax_scale, weight, weight_out, out, lse,
                             workspace)
    B, Hq, T, d = Q.shape
    Hkv, cap = K.shape[1], K.shape[2]
    q = _on(Q, torch.bfloat16, (B, Hq, T, d), "Q", device)
    k, ks = _rows(K, (B, Hkv, cap, d), "K", device)
    v, vs = _rows(V, (B, Hkv, cap, d), "V", device)
    if weight is None and weight_out is not None:
        raise ValueError("weight_out: given without weight")
    if weight is not None and weight_out is None:
        weight_out = weight
    if out is None:
        out = torch.empty_like(Q)
    workspace, ws, ws_bytes = _workspace(workspace, _tree_workspace(B, Hq, Hkv, T, cap, weight is not None), device)
    _check(load().dhsa_tree_attn(
        q, k, ks, v, vs, B, Hq, Hkv, T, cap, d, _on(lengths, torch.int32, (B,), "lengths", device),
        _on(parents, torch.int32, (B, T), "parents", device), _on(n_draft, torch.int32, (B,), "n_draft", device),
        1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale),
        _on(out, torch.bfloat16, (B, Hq, T, d), "out", device), _on(lse, torch.float32, (B, Hq, T), "lse", device),
        _on(weight, torch.float32, (B, Hkv, cap), "weight", device),
        _on(weight_out, torch.float32, (B, Hkv, cap), "weight_out", device), ws, ws_bytes, _raw_stream(device)),
        "dhsa_tree_attn")
    return out


def cache_evict(K: torch.Tensor, V: torch.Tensor, weight: torch.Tensor, pos: torch.Tensor, lengths: torch.Tensor,
                keep: int, next_pos: Optional[torch.Tensor] = None, n_draft: Optional[torch.Tensor] = None,
                accept: Optional[torch.Tensor] = None, sinks: int = 0, recent: int = 0,
                weight_out: Optional[torch.Tensor] = None, pos_out: Optional[torch.Tensor] = None,
                lengths_out: Optional[torch.Tensor] = None, index: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None):
    """Evict all but `keep` slots of each sequence and kv head, in place, and
    commit the accepted drafts (include/dhsa.h, 8).

    weight fp32 and pos int32 [B,Hkv,cap] (updated in place unless weight_out
    and pos_out are given); n_draft int32 [B] drafted slots after `lengths`,
    of which those with their bit in accept (int64 [B]; None: all) may stay.
    Slots with pos < sinks or pos >= next_pos - recent rank first, the lower
    slot first among them if they are more than `keep`. index
    (int32 [B,Hkv,min(keep,cap)]) receives each slot's source.
    Returns lengths_out (a new tensor unless given; not `lengths` itself)."""
    done = (_marshal or _load_marshal()).cache_evict(K, V, weight, pos, lengths, keep, next_pos, n_draft, accept, sinks,
                                                     recent, weight_out, pos_out, lengths_out, index, workspace)
    if done is not None:
        if type(done) is int:
            _check(done, "dhsa_cache_evict")
        return done
    device = _call_device(K, "K")
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return cache_evict(K, V, weight, pos, lengths, keep, next_pos, n_draft, accept, sinks, recent, weight_out,
                               pos_out, lengths_out, index, workspace)
    B, Hkv, cap, d = K.shape
    k, ks = _rows(K, (B, Hkv, cap, d), "K", device)
    v, vs = _rows(V, (B, Hkv, cap, d), "V", device)
    if weight_out is None:
        weight_out = weight
    if pos_out is None:
        pos_out = pos
    if lengths_out is None:
        lengths_out = torch.empty_like(lengths)
    keep, sinks, recent = _int32(keep), _int32(sinks), _int32(recent)
    workspace, ws, ws_bytes = _workspace(workspace, _evict_workspace(B, Hkv, cap), device)
    _check(load().dhsa_cache_evict(
        k, ks, v, vs, _on(weight, torch.float32, (B, Hkv, cap), "weight", device),
        _on(pos, torch.int32, (B, Hkv, cap), "pos", device), B, Hkv, cap, d,
        _on(lengths, torch.int32, (B,), "lengths", device), _on(n_draft, torch.int32, (B,), "n_draft", device),
        _on(accept, torch.int64, (B,), "accept", device), keep, sinks, recent,
        _on(next_pos, torch.int32, (B,), "next_pos", device),
        _on(weight_out, torch.float32, (B, Hkv, cap), "weight_out", device),
        _on(pos_out, torch.int32, (B, Hkv, cap), "pos_out", device),
        _on(lengths_out, torch.int32, (B,), "lengths_out", device),
        _on(index, torch.int32, (B, Hkv, min(keep, cap)), "index", device), ws, ws_bytes, _raw_stream(device)),
        "dhsa_cache_evict")
    return lengths_out


# ----------------------------------------------------------------- whole layer
class DHSAPrefill:
    """The five calls of one DHSA prefill layer with buffers allocated once.

    run(Q, K, V) does pool(Q), pool(K), score + selection, CSR build and
    sparse attention on the current stream and returns O (bf16, like Q).
    Selection is the top-k rule, or, when `budget` is given (an int, or an
    int32 tensor [B, Hq, Nmax] of per-row budgets), the token-budget rule with
    a window of `recent` chunks and at most k earlier chunks per row.
    `short_tiles` picks the query-tile policy of the attention (0: 128-row
    tiles only, the fast default; 1 and 2: see sparse_attn_fwd).
    `fused_routing` runs pooling, the top-k selection and the CSR as one
    launch (route_fused; top-k rule only). Under the top-k rule the selection
    writes the CSR itself (chunk_score_topk_csr); `csr_from_selection=False`
    runs the separate CSR build instead (the same results).
    With `inv_freq` (float64 [rotary_dim/2], see rotary_qkv) run() takes Q and
    K before their rotary positions and rotates them first, at positions
    0 .. L-1, into its own Qr and Kr; Q and K may then be views. Without it
    they are taken as rotated.
    """

    def __init__(self, B: int, Hq: int, Hkv: int, L: int, off: torch.Tensor, n_chunks: torch.Tensor, k: int,
                 device="cuda", softmax_scale: Optional[float] = None, budget=None, recent: int = 0,
                 short_tiles: int = 0, fused_routing: bool = False, csr_from_selection: bool = True,
                 inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False, rotary_factor: float = 1.0):
        lib = load()
        self.B, self.Hq, self.Hkv, self.L, self.k = B, Hq, Hkv, L, k
        self.short_tiles = short_tiles
        if fused_routing and budget is not None:
            raise ValueError("fused_routing supports the top-k rule only")
        self.fused_routing = fused_routing
        self.csr_from_selection = csr_from_selection
        self.budget, self.recent = budget, recent
        self.off, self.n_chunks = off, n_chunks
        self.nmax = off.shape[1] - 1
        nmax = self.nmax
        dev = torch.device(device)
        self.scale = 1.0 / math.sqrt(128) if softmax_scale is None else softmax_scale
        self.Qp = torch.empty((B, Hq, nmax, 128), dtype=torch.float32, device=dev)
        self.Kp = torch.empty((B, Hkv, nmax, 128), dtype=torch.float32, device=dev)
        self.stride = lib.dhsa_sel_stride(k, nmax)
        self.sel = torch.empty((B, Hq, nmax, self.stride), dtype=torch.int32, device=dev)
        self.n_sel = torch.empty((B, Hq, nmax), dtype=torch.int32, device=dev)
        ws1 = lib.dhsa_score_topk_workspace_size(B, Hq, nmax)
        self.ws_topk = torch.empty(max(ws1, 1), dtype=torch.uint8, device=dev) if ws1 else None
        self.row_ptr = torch.empty(B * Hq * nmax + 1, dtype=torch.int32, device=dev)
        self.col_idx = torch.empty(lib.dhsa_csr_nnz_upper(B, Hq, nmax, k), dtype=torch.int32, device=dev)
        self.cost = torch.empty(B * Hq * nmax, dtype=torch.int64, device=dev)
        self.ws_attn = torch.empty(max(lib.dhsa_sparse_attn_tiles_workspace_size(B, Hq, L, nmax, short_tiles), 1),
                                   dtype=torch.uint8, device=dev)
        self.O = torch.empty((B, Hq, L, 128), dtype=torch.bfloat16, device=dev)
        self.inv_freq, self.interleaved, self.rotary_factor = inv_freq, interleaved, rotary_factor
        if inv_freq is not None:
            self.Qr = torch.empty((B, Hq, L, 128), dtype=torch.bfloat16, device=dev)
            self.Kr = torch.empty((B, Hkv, L, 128), dtype=torch.bfloat16, device=dev)

    def rotate(self, Q, K):
        """Q and K at their rotary positions (as they are without inv_freq)."""
        if self.inv_freq is None:
            return Q, K
        rotary_qkv(Q, K, self.inv_freq, interleaved=self.interleaved, factor=self.rotary_factor, Q_out=self.Qr,
                   K_out=self.Kr)
        return self.Qr, self.Kr

    def routing(self, Q, K):
        if self.fused_routing:
            route_fused(Q, K, self.off, self.n_chunks, self.k, Qp=self.Qp, Kp=self.Kp, sel=self.sel,
                        n_sel=self.n_sel, workspace=self.ws_topk, row_ptr=self.row_ptr, col_idx=self.col_idx,
                        cost=self.cost)
            return
        chunk_pool_qk(Q, K, self.off, self.n_chunks, Qp=self.Qp, Kp=self.Kp)
        if self.budget is None and self.csr_from_selection:
            chunk_score_topk_csr(self.Qp, self.Kp, self.off, self.n_chunks, self.k, self.sel, self.n_sel,
                                 self.row_ptr, self.col_idx, cost=self.cost, workspace=self.ws_topk)
            return
        if self.budget is None:
            chunk_score_topk(self.Qp, self.Kp, self.n_chunks, self.k, sel=self.sel, n_sel=self.n_sel,
                             workspace=self.ws_topk)
        else:
            chunk_score_select_budget(self.Qp, self.Kp, self.off, self.n_chunks, self.budget, self.recent, self.k,
                                      sel=self.sel, n_sel=self.n_sel, workspace=self.ws_topk)
        build_block_csr(self.sel, self.n_sel, self.k, self.off, self.n_chunks, row_ptr=self.row_ptr,
                        col_idx=self.col_idx, cost=self.cost)

    def attention(self, Q, K, V):
        return sparse_attn_fwd(Q, K, V, self.off, self.n_chunks, self.row_ptr, self.col_idx, self.cost,
                               self.scale, out=self.O, workspace=self.ws_attn, short_tiles=self.short_tiles)

    def run(self, Q, K, V):
        Q, K = self.rotate(Q, K)
        self.routing(Q, K)
        return self.attention(Q, K, V)


class HostStreamedPrefill:
    """Layers whose Q, K, V arrive in pinned host memory and whose O goes back
    to host memory, one call per layer, with the copies overlapped.

    submit(Qh, Kh, Vh, Oh) enqueues: the host-to-device copy of the layer's
    inputs on a copy-in stream, routing + attention on a compute stream, and
    the device-to-host copy of O on a copy-out stream, chained by events.
    Inputs and outputs are double-buffered on the device, so the copy-in of
    layer s+1 and the copy-out of layer s-1 run while layer s computes (the
    two copy directions use the two PCIe directions). Returns at once;
    synchronize() waits for every submitted layer. Host buffers must stay
    untouched until then.

    A layer with inv_freq keeps its rotated K only until the next one is
    submitted: submit(..., cache=) fills that layer's KVCache with it and V, on
    the compute stream, after what the current stream has done to the cache.
    No other stream may use the cache before synchronize().
    """

    def __init__(self, layer: DHSAPrefill):
        self.layer = layer
        dev = layer.O.device
        B, Hq, Hkv, L = layer.B, layer.Hq, layer.Hkv, layer.L
        self.Qd = [torch.empty((B, Hq, L, 128), dtype=torch.bfloat16, device=dev) for _ in range(2)]
        self.Kd = [torch.empty((B, Hkv, L, 128), dtype=torch.bfloat16, device=dev) for _ in range(2)]
        self.Vd = [torch.empty((B, Hkv, L, 128), dtype=torch.bfloat16, device=dev) for _ in range(2)]
        self.Od = [layer.O, torch.empty_like(layer.O)]
        self.s_in, self.s_comp, self.s_out = (torch.cuda.Stream(dev) for _ in range(3))
        self.e_in = [torch.cuda.Event() for _ in range(2)]
        self.e_comp = [torch.cuda.Event() for _ in range(2)]
        self.e_out = [torch.cuda.Event() for _ in range(2)]
        self.n = 0

    def submit(self, Qh: torch.Tensor, Kh: torch.Tensor, Vh: torch.Tensor, Oh: torch.Tensor, cache=None):
        b = self.n & 1
        lay = self.layer
        if self.n >= 2:
            self.s_in.wait_event(self.e_comp[b])       # layer n-2 has read this input set
        with torch.cuda.stream(self.s_in):
            self.Qd[b].copy_(Qh, non_blocking=True)
            self.Kd[b].copy_(Kh, non_blocking=True)
            self.Vd[b].copy_(Vh, non_blocking=True)
            self.e_in[b].record(self.s_in)
        self.s_comp.wait_event(self.e_in[b])
        if self.n >= 2:
            self.s_comp.wait_event(self.e_out[b])      # layer n-2's O has left this buffer
        if cache is not None:
            self.s_comp.wait_stream(torch.cuda.current_stream(self.s_comp.device))
        with torch.cuda.stream(self.s_comp):
            Q, K = lay.rotate(self.Qd[b], self.Kd[b])
            if cache is not None:
                cache.fill(K, self.Vd[b])
            lay.routing(Q, K)
            sparse_attn_fwd(Q, K, self.Vd[b], lay.off, lay.n_chunks, lay.row_ptr, lay.col_idx,
                            lay.cost, lay.scale, out=self.Od[b], workspace=lay.ws_attn)
            self.e_comp[b].record(self.s_comp)
        self.s_out.wait_event(self.e_comp[b])
        with torch.cuda.stream(self.s_out):
            Oh.copy_(self.Od[b], non_blocking=True)
            self.e_out[b].record(self.s_out)
        self.n += 1

    def synchronize(self):
        for s in (self.s_in, self.s_comp, self.s_out):
            s.synchronize()


class GraphedPrefill:
    """One DHSA layer captured as a CUDA graph: the eight launches of
    DHSAPrefill.run replayed with one graph launch.

    Q, K, V are the device tensors the graph reads; refill them in place and
    call replay(), which returns the layer's O tensor (the same buffer each
    time). The chunk offsets and the selection settings are those of `layer`
    at capture time.
    """

    def __init__(self, layer: DHSAPrefill, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor):
        self.layer, self.Q, self.K, self.V = layer, Q, K, V
        s = torch.cuda.Stream(Q.device)
        s.wait_stream(torch.cuda.current_stream(Q.device))
        with torch.cuda.stream(s):              # one eager run first (module load, function attributes)
            layer.run(Q, K, V)
        torch.cuda.current_stream(Q.device).wait_stream(s)
        torch.cuda.synchronize(Q.device)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.O = layer.run(Q, K, V)

    def replay(self) -> torch.Tensor:
        self.graph.replay()
        return self.O
