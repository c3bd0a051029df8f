"""Thin Python binding of libssd (the C ABI in include/ssd.h).

Argument marshalling only: tensors are checked for device/dtype/contiguity, turned into raw
pointers and passed with torch's current CUDA stream.  Every step of the computation runs in the
CUDA kernels of libssd.so; there is no fallback.  If the library has not been built, every call
raises ``LibraryNotBuilt`` -- build it with ``sparse_self_speculative_verify_gb300.build.build()``.

PyTorch supplies device memory (outputs and zero-initialised workspaces) and streams.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading
from dataclasses import dataclass
from typing import Optional

import torch

from . import build as _build

SSD_OK, SSD_ERR_INVALID_ARG, SSD_ERR_UNSUPPORTED, SSD_ERR_WORKSPACE, SSD_ERR_CUDA, SSD_ERR_TIMEOUT = range(6)
SSD_DTYPE_F32, SSD_DTYPE_BF16, SSD_DTYPE_NVFP4 = 0, 1, 2
FAULT_PAGE, FAULT_SEQLEN, FAULT_INDEX, FAULT_KMAX, FAULT_UNION, FAULT_TIMEOUT, FAULT_VALUE, FAULT_NOPAGE = \
    1, 2, 4, 8, 16, 32, 64, 128

EXPORTED = ["ssd_last_error", "ssd_version", "ssd_status", "ssd_verify_workspace_bytes", "ssd_verify_attn",
            "ssd_verify_select", "ssd_verify_select_packed",
            "ssd_select_topk", "ssd_select_topp", "ssd_draft_workspace_bytes", "ssd_draft_attn", "ssd_draft_attn_static",
            "ssd_draft_pack_bytes", "ssd_draft_attn_packed",
            "ssd_unified_workspace_bytes", "ssd_kv_append", "ssd_kv_advance", "ssd_phase_assign", "ssd_phase_fill",
            "ssd_unified_attn", "ssd_block_union", "ssd_block_sparse_workspace_bytes", "ssd_block_sparse_attn",
            "ssd_combine",
            "ssd_kv4_append", "ssd_kv4_read", "ssd_kv4_verify_workspace_bytes", "ssd_kv4_verify_attn",
            "ssd_kv4_draft_workspace_bytes", "ssd_kv4_draft_attn",
            "ssd_kv_fork", "ssd_kv_reserve_workspace_bytes", "ssd_kv_reserve", "ssd_kv_release", "ssd_kv_compact",
            "ssd_tree_workspace_bytes", "ssd_tree_attn", "ssd_window_workspace_bytes", "ssd_window_attn",
            "ssd_token_logprobs", "ssd_tree_accept", "ssd_tree_commit"]


class LibraryNotBuilt(RuntimeError):
    pass


class SSDError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class PagedKVStruct(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("dtype", ctypes.c_int), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int), ("h_kv", ctypes.c_int), ("d", ctypes.c_int),
                ("page_table", ctypes.c_void_p), ("max_pages", ctypes.c_int), ("seq_lens", ctypes.c_void_p),
                ("batch", ctypes.c_int), ("max_seq_len", ctypes.c_int)]


_LIB = None
_LOCK = threading.Lock()


def library_path() -> str:
    return _build.lib_path()


def load(path: Optional[str] = None, as_default: bool = False):
    """Load libssd.so (no build step).  Raises LibraryNotBuilt when it is missing.  A library given
    by ``path`` serves the calls of this module only with ``as_default``."""
    global _LIB
    with _LOCK:
        if _LIB is not None and path is None:
            return _LIB
        p = path or library_path()
        if not os.path.exists(p):
            raise LibraryNotBuilt(f"{p} does not exist; build it with sparse_self_speculative_verify_gb300.build.build()")
        L = ctypes.CDLL(p)
        P, I, I64, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        D = ctypes.c_double
        KV = ctypes.POINTER(PagedKVStruct)
        sig = {
            "ssd_last_error": ([], ctypes.c_char_p),
            "ssd_version": ([], I),
            "ssd_status": ([P, ctypes.POINTER(ctypes.c_uint32)], I),
            "ssd_verify_workspace_bytes": ([KV, I, I], S),
            "ssd_verify_attn": ([KV, P, I, I, F, P, P, P, I64, P, I64, I, P, S, P], I),
            "ssd_verify_select": ([KV, P, I, I, F, P, P, P, I64, P, P, I, P, P, S, P], I),
            "ssd_verify_select_packed": ([KV, P, I, I, F, P, P, P, I64, P, P, I, P, P, S, P, S, P], I),
            "ssd_select_topk": ([P, I64, P, P, I, I, I, I, P, I, P, P], I),
            "ssd_select_topp": ([P, I64, P, F, I, I, I, I, P, I, P, P, P], I),
            "ssd_draft_workspace_bytes": ([KV, I, I], S),
            "ssd_draft_attn": ([KV, P, I, P, I, P, F, P, P, P, S, P], I),
            "ssd_draft_attn_static": ([KV, P, I, P, I, P, F, P, P, P], I),
            "ssd_draft_pack_bytes": ([KV, I], S),
            "ssd_draft_attn_packed": ([KV, P, I, P, I, P, F, P, P, P, S, I, P, S, P], I),
            "ssd_kv_append": ([KV, P, P, I, P], I),
            "ssd_kv_advance": ([P, P, I, I, P], I),
            "ssd_phase_assign": ([P, I, I, P], I),
            "ssd_phase_fill": ([P, I, I, I64, P, P], I),
            "ssd_unified_workspace_bytes": ([KV, I, I, I], S),
            "ssd_unified_attn": ([KV, P, P, P, I, I, P, I, P, F, P, P, P, I64, P, P, P, S, P], I),
            "ssd_block_union": ([P, P, I, I, I, I, P, P, P, I, P], I),
            "ssd_block_sparse_workspace_bytes": ([KV, I, I, I], S),
            "ssd_block_sparse_attn": ([KV, P, I, I, P, P, P, I, I, F, P, P, P, S, P], I),
            "ssd_combine": ([P, P, I, I, I, P, P, P], I),
            "ssd_kv4_append": ([KV, P, P, I, I, P, F, F, P], I),
            "ssd_kv4_read": ([KV, P, P, I, F, F, I, P, P, P], I),
            "ssd_kv4_verify_workspace_bytes": ([KV, I, I], S),
            "ssd_kv4_verify_attn": ([KV, P, I, I, I, F, F, F, P, I, P, P, I64, P, S, P], I),
            "ssd_kv4_draft_workspace_bytes": ([KV, I, I], S),
            "ssd_kv_fork": ([KV, P, P, P, I, P], I),
            "ssd_kv_reserve_workspace_bytes": ([KV], S),
            "ssd_kv_reserve": ([KV, P, P, P, S, P], I),
            "ssd_kv_release": ([KV, P, P, P], I),
            "ssd_kv_compact": ([KV, KV, P, P, P, I, P, I, P, P], I),
            "ssd_tree_workspace_bytes": ([KV, I, I], S),
            "ssd_tree_attn": ([KV, P, I, I, P, P, F, P, P, P, S, P], I),
            "ssd_window_workspace_bytes": ([KV, I, I, I, I], S),
            "ssd_window_attn": ([KV, P, I, I, P, I, I, F, P, P, P, S, P], I),
            "ssd_token_logprobs": ([P, I, I64, I, I, P, P, I, P, P, P, P, P, I, P], I),
            "ssd_tree_accept": ([P, P, P, P, P, D, D, P, I, I, I, P, P, P, P, P], I),
            "ssd_tree_commit": ([KV, I, P, P, I, P, P], I),
            "ssd_kv4_draft_attn": ([KV, P, I, I, P, I, P, F, F, F, P, I, P, P, S, P], I),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        if path is None or as_default:
            _LIB = L
        return L


def _lib():
    return _LIB if _LIB is not None else load()


def _check(rc: int):
    if rc != SSD_OK:
        raise SSDError(rc, _lib().ssd_last_error().decode(errors="replace"))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


# ------------------------------------------------------------------------------------------------
# Paged KV cache handle and workspaces.
# ------------------------------------------------------------------------------------------------


@dataclass
class KVCache:
    """pool [num_pages, 2, h_kv, page_size, d] (bf16 or fp32), page_table [B, max_pages] int32,
    seq_lens [B] int32, max_seq_len (host int, >= every seq_len)."""
    pool: torch.Tensor
    page_table: torch.Tensor
    seq_lens: torch.Tensor
    max_seq_len: int

    def __post_init__(self):
        _need(self.pool, "pool")
        _need(self.page_table, "page_table", torch.int32, self.pool.device)
        _need(self.seq_lens, "seq_lens", torch.int32, self.pool.device)
        if self.pool.dim() != 5 or self.pool.shape[1] != 2:
            raise ValueError("pool must be [num_pages, 2, h_kv, page_size, d]")
        if self.pool.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("pool must be bf16 or fp32")
        self._struct = PagedKVStruct(
            self.pool.data_ptr(), SSD_DTYPE_BF16 if self.pool.dtype == torch.bfloat16 else SSD_DTYPE_F32,
            self.pool.shape[0], self.pool.shape[3], self.pool.shape[2], self.pool.shape[4],
            self.page_table.data_ptr(), self.page_table.shape[1], self.seq_lens.data_ptr(),
            self.seq_lens.shape[0], int(self.max_seq_len))
        self._geometry = (self.pool.get_device(), self.batch, self.h_kv, self.d)
        self._ref = ctypes.byref(self._struct)
        self._need = {}  # workspace bytes of the tree and window calls' shapes

    @property
    def h_kv(self) -> int:
        return self.pool.shape[2]

    @property
    def d(self) -> int:
        return self.pool.shape[4]

    @property
    def batch(self) -> int:
        return self.seq_lens.shape[0]

    @property
    def device(self):
        return self.pool.device

    def ref(self):
        return self._ref

    @classmethod
    def from_workload(cls, w) -> "KVCache":
        return cls(w.pool, w.page_table, w.seq_lens, w.max_seq_len)


COUNTER_BYTES = 1 << 18  # the counter area at a workspace's start


class Workspace:
    """Zero-initialised device scratch buffers, grown on demand, one per (device, name).  The
    library keeps its counters in a fixed area at the start of a workspace and returns them to zero
    after each call, so a buffer is zeroed only once and serves calls of any shape in turn."""

    def __init__(self):
        self._bufs = {}
        self._captured = []  # buffers that graphs captured from the 4-bit and page calls hold: kept when others replace them

    def get(self, device, name: str, nbytes: int) -> torch.Tensor:
        key = (str(device), name)
        buf = self._bufs.get(key)
        if buf is None or buf.numel() < nbytes:
            buf = torch.zeros(max(int(nbytes), 256) + 256, dtype=torch.uint8, device=device)
            self._bufs[key] = buf
        return buf

    @staticmethod
    def aligned(buf: torch.Tensor) -> int:
        p = buf.data_ptr()
        return (p + 255) & ~255


_DEFAULT_WS = Workspace()


def _ws(kv_device, name, nbytes, workspace: Optional[Workspace]):
    ws = (workspace or _DEFAULT_WS).get(kv_device, name, nbytes)
    base = Workspace.aligned(ws)
    avail = ws.data_ptr() + ws.numel() - base
    return ctypes.c_void_p(base), avail


# ------------------------------------------------------------------------------------------------
# Calls (same names as the C ABI).
# ------------------------------------------------------------------------------------------------


def ssd_version() -> int:
    return _lib().ssd_version()


def ssd_status(stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check(_lib().ssd_status(_stream(stream), ctypes.byref(v)))
    return v.value


def ssd_verify_attn(kv: KVCache, q: torch.Tensor, n_cand: int, scale: float, *, out=None, lse=None,
                    scores: Optional[torch.Tensor] = None, bscores: Optional[torch.Tensor] = None,
                    block_size: int = 64, want_scores: bool = True, want_lse: bool = True,
                    workspace: Optional[Workspace] = None, stream=None) -> dict:
    """Verify attention over the paged cache with fused criticality.  q [B, n_cand, h_q, d]."""
    _need(q, "q", kv.pool.dtype, kv.device)
    B, nc, h_q, d = q.shape
    assert nc == n_cand and B == kv.batch and d == kv.d
    dev = kv.device
    if out is None:
        out = torch.empty((B, nc, h_q, d), dtype=torch.float32, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((B, nc, h_q), dtype=torch.float32, device=dev)
    if scores is None and want_scores:
        scores = torch.zeros((B, kv.h_kv, max(kv.max_seq_len, 1)), dtype=torch.float32, device=dev)
    for t, n in ((out, "out"), (lse, "lse"), (scores, "scores"), (bscores, "bscores")):
        if t is not None:
            _need(t, n, torch.float32, dev)
    L = _lib()
    need = L.ssd_verify_workspace_bytes(kv.ref(), h_q, n_cand)
    wsp, avail = _ws(dev, "verify", need, workspace)
    _check(L.ssd_verify_attn(kv.ref(), _ptr(q), h_q, n_cand, float(scale), _ptr(out), _ptr(lse), _ptr(scores),
                             scores.shape[-1] if scores is not None else 0, _ptr(bscores),
                             bscores.shape[-1] if bscores is not None else 0, block_size, wsp, avail,
                             _stream(stream)))
    return {"out": out, "lse": lse, "scores": scores, "bscores": bscores}


def ssd_verify_select(kv: KVCache, q: torch.Tensor, n_cand: int, scale: float, ks: torch.Tensor, k_max: int, *,
                      out=None, lse=None, scores=None, idx=None, cnt=None, want_lse: bool = True,
                      pack: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None,
                      stream=None) -> dict:
    """Verify with the Top-K selection fused into its criticality pass.  q [B, n_cand, h_q, d];
    ks [B] int32 (K per request); idx [B * h_kv, k_max], cnt [B * h_kv].  With `pack` (a uint8 buffer
    of ssd_draft_pack_bytes(kv, k_max) bytes, 256-byte aligned), ssd_verify_select_packed: the
    selected rows are also stored there for drafts with PACK_READ."""
    _need(q, "q", kv.pool.dtype, kv.device)
    B, nc, h_q, d = q.shape
    assert nc == n_cand and B == kv.batch and d == kv.d
    dev = kv.device
    _need(ks, "ks", torch.int32, dev)
    if out is None:
        out = torch.empty((B, nc, h_q, d), dtype=torch.float32, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((B, nc, h_q), dtype=torch.float32, device=dev)
    if scores is None:
        scores = torch.zeros((B, kv.h_kv, max(kv.max_seq_len, 1)), dtype=torch.float32, device=dev)
    if idx is None:
        idx = torch.empty((B * kv.h_kv, max(k_max, 0)), dtype=torch.int32, device=dev)
    if cnt is None:
        cnt = torch.empty((B * kv.h_kv,), dtype=torch.int32, device=dev)
    for t, n, dt in ((out, "out", torch.float32), (lse, "lse", torch.float32), (scores, "scores", torch.float32),
                     (idx, "idx", torch.int32), (cnt, "cnt", torch.int32)):
        if t is not None:
            _need(t, n, dt, dev)
    L = _lib()
    need = L.ssd_verify_workspace_bytes(kv.ref(), h_q, n_cand)
    wsp, avail = _ws(dev, "verify", need, workspace)
    if pack is None:
        _check(L.ssd_verify_select(kv.ref(), _ptr(q), h_q, n_cand, float(scale), _ptr(out), _ptr(lse), _ptr(scores),
                                   scores.shape[-1], _ptr(ks), _ptr(idx), k_max, _ptr(cnt), wsp, avail,
                                   _stream(stream)))
    else:
        _need(pack, "pack", torch.uint8, dev)
        _check(L.ssd_verify_select_packed(kv.ref(), _ptr(q), h_q, n_cand, float(scale), _ptr(out), _ptr(lse),
                                          _ptr(scores), scores.shape[-1], _ptr(ks), _ptr(idx), k_max, _ptr(cnt),
                                          _ptr(pack), pack.numel(), wsp, avail, _stream(stream)))
    return {"out": out, "lse": lse, "scores": scores, "idx": idx, "cnt": cnt}


def ssd_select_topk(scores: torch.Tensor, lens: torch.Tensor, ks: torch.Tensor, k_max: int, rows_per_group: int,
                    len_div: int = 1, max_len: Optional[int] = None, *, idx=None, cnt=None, stream=None):
    """Top-K per row of a [n_rows, stride] (or [..., stride]) fp32 score tensor."""
    _need(scores, "scores", torch.float32)
    dev = scores.device
    _need(lens, "lens", torch.int32, dev)
    _need(ks, "ks", torch.int32, dev)
    stride = scores.shape[-1]
    n_rows = scores.numel() // stride
    n_groups = lens.shape[0]
    assert n_groups * rows_per_group == n_rows and ks.shape[0] == n_groups
    if max_len is None:
        max_len = stride
    if idx is None:
        idx = torch.empty((n_rows, max(k_max, 0)), dtype=torch.int32, device=dev)
    if cnt is None:
        cnt = torch.empty((n_rows,), dtype=torch.int32, device=dev)
    _need(idx, "idx", torch.int32, dev)
    _need(cnt, "cnt", torch.int32, dev)
    _check(_lib().ssd_select_topk(_ptr(scores), stride, _ptr(lens), _ptr(ks), n_groups, rows_per_group, len_div,
                                  int(max_len), _ptr(idx), k_max, _ptr(cnt), _stream(stream)))
    return idx, cnt


def ssd_select_topp(scores: torch.Tensor, lens: torch.Tensor, p: float, k_max: int, rows_per_group: int,
                    len_div: int = 1, max_len: Optional[int] = None, *, idx=None, cnt=None, k_rows=None,
                    stream=None):
    """Top-p per row: the fewest largest entries whose sum reaches p times the row total, at most
    k_max.  Returns (idx, cnt, k_rows); k_rows is the per-row count before the Top-K pass."""
    _need(scores, "scores", torch.float32)
    dev = scores.device
    _need(lens, "lens", torch.int32, dev)
    stride = scores.shape[-1]
    n_rows = scores.numel() // stride
    n_groups = lens.shape[0]
    assert n_groups * rows_per_group == n_rows
    if max_len is None:
        max_len = stride
    if idx is None:
        idx = torch.empty((n_rows, max(k_max, 0)), dtype=torch.int32, device=dev)
    if cnt is None:
        cnt = torch.empty((n_rows,), dtype=torch.int32, device=dev)
    if k_rows is None:
        k_rows = torch.empty((n_rows,), dtype=torch.int32, device=dev)
    for t, name in ((idx, "idx"), (cnt, "cnt"), (k_rows, "k_rows")):
        _need(t, name, torch.int32, dev)
    _check(_lib().ssd_select_topp(_ptr(scores), stride, _ptr(lens), float(p), n_groups, rows_per_group, len_div,
                                  int(max_len), _ptr(idx), k_max, _ptr(cnt), _ptr(k_rows), _stream(stream)))
    return idx, cnt, k_rows


def ssd_draft_attn(kv: KVCache, q: torch.Tensor, idx: torch.Tensor, cnt: torch.Tensor, scale: float, *, out=None,
                   lse=None, want_lse: bool = True, workspace: Optional[Workspace] = None, stream=None) -> dict:
    """Single-query attention over the selected tokens.  q [B, h_q, d]; idx [B, h_kv, k_max]."""
    _need(q, "q", kv.pool.dtype, kv.device)
    dev = kv.device
    _need(idx, "idx", torch.int32, dev)
    _need(cnt, "cnt", torch.int32, dev)
    B, h_q, d = q.shape
    k_max = idx.shape[-1]
    if out is None:
        out = torch.empty((B, h_q, d), dtype=torch.float32, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((B, h_q), dtype=torch.float32, device=dev)
    L = _lib()
    need = L.ssd_draft_workspace_bytes(kv.ref(), h_q, k_max)
    wsp, avail = _ws(dev, "draft", need, workspace)
    _check(L.ssd_draft_attn(kv.ref(), _ptr(q), h_q, _ptr(idx), k_max, _ptr(cnt), float(scale), _ptr(out), _ptr(lse),
                            wsp, avail, _stream(stream)))
    return {"out": out, "lse": lse}


PACK_NONE, PACK_WRITE, PACK_READ, PACK_READ_DISCARD = 0, 1, 2, 3


def ssd_draft_pack_bytes(kv: KVCache, k_max: int) -> int:
    return int(_lib().ssd_draft_pack_bytes(kv.ref(), int(k_max)))


def ssd_draft_attn_packed(kv: KVCache, q: torch.Tensor, idx: Optional[torch.Tensor], cnt: torch.Tensor, scale: float,
                          pack: torch.Tensor, pack_mode: int, *, k_max: Optional[int] = None, out=None, lse=None,
                          want_lse: bool = True, workspace: Optional[Workspace] = None, stream=None) -> dict:
    """ssd_draft_attn with a row pack: PACK_WRITE attends through idx and stores the selected rows in
    ``pack`` (a uint8 device tensor of ssd_draft_pack_bytes bytes, 256-byte aligned); PACK_READ
    attends the rows stored by the last PACK_WRITE call (idx may be None; then k_max is required);
    PACK_READ_DISCARD reads likewise and leaves the pack undefined (the round's last draft: its lines
    leave L2 without being written back)."""
    _need(q, "q", kv.pool.dtype, kv.device)
    dev = kv.device
    if idx is not None:
        _need(idx, "idx", torch.int32, dev)
    _need(cnt, "cnt", torch.int32, dev)
    _need(pack, "pack", torch.uint8, dev)
    B, h_q, d = q.shape
    if k_max is None:
        if idx is None:
            raise ValueError("k_max is required when idx is None")
        k_max = idx.shape[-1]
    if out is None:
        out = torch.empty((B, h_q, d), dtype=torch.float32, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((B, h_q), dtype=torch.float32, device=dev)
    L = _lib()
    need = L.ssd_draft_workspace_bytes(kv.ref(), h_q, k_max)
    wsp, avail = _ws(dev, "draft", need, workspace)
    _check(L.ssd_draft_attn_packed(kv.ref(), _ptr(q), h_q, _ptr(idx), int(k_max), _ptr(cnt), float(scale), _ptr(out),
                                   _ptr(lse), _ptr(pack), pack.numel(), int(pack_mode), wsp, avail, _stream(stream)))
    return {"out": out, "lse": lse}


def ssd_draft_attn_static(kv: KVCache, q: torch.Tensor, idx: torch.Tensor, cnt: torch.Tensor, scale: float, *,
                          out=None, lse=None, want_lse: bool = True, stream=None) -> dict:
    """ssd_draft_attn without a workspace: the scratch is the library's built-in device array
    (SSD_DRAFT_STATIC_SCRATCH_BYTES), so nothing is allocated for it.  For callers that cannot
    allocate device memory where they run the draft step.  Calls that can overlap on the GPU share
    that array and race; the first call on a device must come before any stream capture there."""
    _need(q, "q", kv.pool.dtype, kv.device)
    dev = kv.device
    _need(idx, "idx", torch.int32, dev)
    _need(cnt, "cnt", torch.int32, dev)
    B, h_q, d = q.shape
    k_max = idx.shape[-1]
    if out is None:
        out = torch.empty((B, h_q, d), dtype=torch.float32, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((B, h_q), dtype=torch.float32, device=dev)
    _check(_lib().ssd_draft_attn_static(kv.ref(), _ptr(q), h_q, _ptr(idx), k_max, _ptr(cnt), float(scale), _ptr(out),
                                        _ptr(lse), _stream(stream)))
    return {"out": out, "lse": lse}


def ssd_kv_append(kv: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
    """Writes k_new / v_new [B, n_new, h_kv, d] (the pool's dtype) at positions seq_lens[b] + j of
    every request; kv.pool is modified in place, kv.seq_lens is not."""
    _need(k_new, "k_new", kv.pool.dtype, kv.device)
    _need(v_new, "v_new", kv.pool.dtype, kv.device)
    if k_new.shape != v_new.shape or k_new.dim() != 4 or k_new.shape[0] != kv.batch or \
            k_new.shape[2] != kv.h_kv or k_new.shape[3] != kv.d:
        raise ValueError("k_new and v_new must both be [batch, n_new, h_kv, d]")
    _check(_lib().ssd_kv_append(kv.ref(), _ptr(k_new), _ptr(v_new), k_new.shape[1], _stream(stream)))


def ssd_kv_advance(seq_lens: torch.Tensor, delta: torch.Tensor, max_seq_len: int, stream=None) -> None:
    """seq_lens += delta in place on the device (results outside [0, max_seq_len] are left as they
    were and flagged in the device status)."""
    _need(seq_lens, "seq_lens", torch.int32, seq_lens.device)
    _need(delta, "delta", torch.int32, seq_lens.device)
    if delta.shape != seq_lens.shape:
        raise ValueError("delta must have the shape of seq_lens")
    _check(_lib().ssd_kv_advance(_ptr(seq_lens), _ptr(delta), seq_lens.shape[0], int(max_seq_len),
                                 _stream(stream)))


def ssd_phase_assign(counts, n_new: int):
    """Greedy phase offsets for n_new arriving requests.  counts: host int32 array [k + 1] of live
    requests per offset (numpy or CPU tensor), updated in place; returns the offsets (int32 numpy)."""
    import numpy as np
    c = counts.numpy() if isinstance(counts, torch.Tensor) else counts
    if not isinstance(c, np.ndarray) or c.dtype != np.int32 or not c.flags["C_CONTIGUOUS"]:
        raise TypeError("counts must be a contiguous int32 host array")
    out = np.zeros(max(n_new, 1), np.int32)
    _check(_lib().ssd_phase_assign(c.ctypes.data_as(ctypes.c_void_p), c.shape[0], int(n_new),
                                   out.ctypes.data_as(ctypes.c_void_p)))
    return out[:n_new]


def ssd_phase_fill(offsets: torch.Tensor, n_buckets: int, step: int, *, phase=None, stream=None) -> torch.Tensor:
    """Device phase array for ssd_unified_attn at `step`: 1 = verify, 0 = draft."""
    _need(offsets, "offsets", torch.int32, offsets.device)
    if phase is None:
        phase = torch.empty(offsets.shape, dtype=torch.uint8, device=offsets.device)
    _need(phase, "phase", torch.uint8, offsets.device)
    _check(_lib().ssd_phase_fill(_ptr(offsets), offsets.shape[0], int(n_buckets), int(step), _ptr(phase),
                                 _stream(stream)))
    return phase


def ssd_unified_attn(kv: KVCache, phase: torch.Tensor, q_verify: torch.Tensor, q_draft: torch.Tensor, n_cand: int,
                     idx: torch.Tensor, cnt: torch.Tensor, scale: float, *, out_verify=None, lse_verify=None,
                     scores=None, out_draft=None, lse_draft=None, want_scores: bool = True,
                     workspace: Optional[Workspace] = None, stream=None) -> dict:
    """Mixed batch: verify-phase requests (phase == 1) get verify + criticality, draft-phase requests
    (phase == 0) the sparse draft, in one call."""
    dev = kv.device
    _need(phase, "phase", torch.uint8, dev)
    _need(q_verify, "q_verify", kv.pool.dtype, dev)
    _need(q_draft, "q_draft", kv.pool.dtype, dev)
    _need(idx, "idx", torch.int32, dev)
    _need(cnt, "cnt", torch.int32, dev)
    B, nc, h_q, d = q_verify.shape
    k_max = idx.shape[-1]
    if out_verify is None:
        out_verify = torch.zeros((B, nc, h_q, d), dtype=torch.float32, device=dev)
    if lse_verify is None:
        lse_verify = torch.zeros((B, nc, h_q), dtype=torch.float32, device=dev)
    if scores is None and want_scores:
        scores = torch.zeros((B, kv.h_kv, max(kv.max_seq_len, 1)), dtype=torch.float32, device=dev)
    if out_draft is None:
        out_draft = torch.zeros((B, h_q, d), dtype=torch.float32, device=dev)
    if lse_draft is None:
        lse_draft = torch.zeros((B, h_q), dtype=torch.float32, device=dev)
    L = _lib()
    need = L.ssd_unified_workspace_bytes(kv.ref(), h_q, n_cand, k_max)
    wsp, avail = _ws(dev, "unified", need, workspace)
    _check(L.ssd_unified_attn(kv.ref(), _ptr(phase), _ptr(q_verify), _ptr(q_draft), h_q, n_cand, _ptr(idx), k_max,
                              _ptr(cnt), float(scale), _ptr(out_verify), _ptr(lse_verify), _ptr(scores),
                              scores.shape[-1] if scores is not None else 0, _ptr(out_draft), _ptr(lse_draft), wsp,
                              avail, _stream(stream)))
    return {"out_verify": out_verify, "lse_verify": lse_verify, "scores": scores, "out_draft": out_draft,
            "lse_draft": lse_draft}


def ssd_block_union(blocks: torch.Tensor, bcnt: torch.Tensor, nblk_max: int, umax: Optional[int] = None, *,
                    uidx=None, umask=None, ucnt=None, stream=None):
    """Union of the candidates' block sets.  blocks [units, n_cand, kb], bcnt [units, n_cand]."""
    _need(blocks, "blocks", torch.int32)
    dev = blocks.device
    _need(bcnt, "bcnt", torch.int32, dev)
    U, nc, kb = blocks.shape
    um = umax or nc * kb
    if uidx is None:
        uidx = torch.empty((U, um), dtype=torch.int32, device=dev)
    if umask is None:
        umask = torch.empty((U, um), dtype=torch.int32, device=dev)  # uint32 bit patterns
    if ucnt is None:
        ucnt = torch.empty((U,), dtype=torch.int32, device=dev)
    _need(uidx, "uidx", torch.int32, dev)
    _need(umask, "umask", torch.int32, dev)
    _need(ucnt, "ucnt", torch.int32, dev)
    assert uidx.shape == (U, um) and umask.shape == (U, um) and ucnt.shape == (U,)
    _check(_lib().ssd_block_union(_ptr(blocks), _ptr(bcnt), U, nc, kb, nblk_max, _ptr(uidx), _ptr(umask), _ptr(ucnt),
                                  um, _stream(stream)))
    return uidx, umask, ucnt


def ssd_block_sparse_attn(kv: KVCache, q: torch.Tensor, n_cand: int, uidx: torch.Tensor, umask: torch.Tensor,
                          ucnt: torch.Tensor, scale: float, block_size: int = 64, *, out=None, lse=None,
                          workspace: Optional[Workspace] = None, stream=None) -> dict:
    """Block-sparse attention of the candidates over their union blocks (each loaded once)."""
    dev = kv.device
    _need(q, "q", kv.pool.dtype, dev)
    _need(uidx, "uidx", torch.int32, dev)
    _need(umask, "umask", torch.int32, dev)
    _need(ucnt, "ucnt", torch.int32, dev)
    B, nc, h_q, d = q.shape
    umax = uidx.shape[-1]
    if out is None:
        out = torch.empty((B, nc, h_q, d), dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty((B, nc, h_q), dtype=torch.float32, device=dev)
    L = _lib()
    need = L.ssd_block_sparse_workspace_bytes(kv.ref(), h_q, n_cand, umax)
    wsp, avail = _ws(dev, "block", need, workspace)
    _check(L.ssd_block_sparse_attn(kv.ref(), _ptr(q), h_q, n_cand, _ptr(uidx), _ptr(umask), _ptr(ucnt), umax,
                                   block_size, float(scale), _ptr(out), _ptr(lse), wsp, avail, _stream(stream)))
    return {"out": out, "lse": lse}


def ssd_combine(o_parts: torch.Tensor, lse_parts: torch.Tensor, *, out=None, lse=None, stream=None):
    """LSE merge of split partials: o_parts [rows, splits, d], lse_parts [rows, splits]."""
    _need(o_parts, "o_parts", torch.float32)
    dev = o_parts.device
    _need(lse_parts, "lse_parts", torch.float32, dev)
    R, S, d = o_parts.shape
    if out is None:
        out = torch.empty((R, d), dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty((R,), dtype=torch.float32, device=dev)
    _check(_lib().ssd_combine(_ptr(o_parts), _ptr(lse_parts), R, S, d, _ptr(out), _ptr(lse), _stream(stream)))
    return out, lse


# ------------------------------------------------------------------------------------------------
# 4-bit paged cache (NVFP4).
# ------------------------------------------------------------------------------------------------


@dataclass
class KV4Cache:
    """A 4-bit paged cache: pool uint8 [num_pages, 2, h_kv, page_size, d / 2 + d / 16] (the shape sizes a
    page's blocks; inside one, all tokens' codes come before their scales), page_table [B, max_pages]
    int32, seq_lens [B] int32, max_seq_len (host int, >= every seq_len), and the power-of-two factors that
    stored K and V values are multiplied with.  ``pool_shape`` gives the shape to allocate."""
    pool: torch.Tensor
    page_table: torch.Tensor
    seq_lens: torch.Tensor
    max_seq_len: int
    k_scale: float = 1.0
    v_scale: float = 1.0

    def __post_init__(self):
        _need(self.pool, "pool", torch.uint8)
        _need(self.page_table, "page_table", torch.int32, self.pool.device)
        _need(self.seq_lens, "seq_lens", torch.int32, self.pool.device)
        if self.pool.dim() != 5 or self.pool.shape[1] != 2 or self.pool.shape[4] not in (36, 72):
            raise ValueError("pool must be [num_pages, 2, h_kv, page_size, d / 2 + d / 16] with d 64 or 128")
        if self.seq_lens.dim() != 1 or self.page_table.dim() != 2 or self.page_table.shape[0] != self.seq_lens.shape[0]:
            raise ValueError("page_table must be [batch, max_pages] and seq_lens [batch]")
        self._struct = PagedKVStruct(
            self.pool.data_ptr(), SSD_DTYPE_NVFP4, self.pool.shape[0], self.pool.shape[3], self.pool.shape[2], self.d,
            self.page_table.data_ptr(), self.page_table.shape[1], self.seq_lens.data_ptr(), self.seq_lens.shape[0],
            int(self.max_seq_len))
        self.k_scale, self.v_scale = float(self.k_scale), float(self.v_scale)
        self._geometry = (self.pool.get_device(), self.batch, self.h_kv, self.d)
        self._ref = ctypes.byref(self._struct)
        self._need = {}  # workspace bytes of the calls' shapes

    @staticmethod
    def pool_shape(num_pages: int, h_kv: int, page_size: int, d: int):
        return (num_pages, 2, h_kv, page_size, d // 2 + d // 16)

    @property
    def h_kv(self) -> int:
        return self.pool.shape[2]

    @property
    def d(self) -> int:
        return self.pool.shape[4] * 16 // 9

    @property
    def batch(self) -> int:
        return self.seq_lens.shape[0]

    @property
    def device(self):
        return self.pool.device

    def ref(self):
        return self._ref


def _c_int(v, name: str) -> int:
    """A whole number that a C int holds (ctypes would keep its low 32 bits)."""
    v = int(v)
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"{name} {v} out of range")
    return v


_empty = torch.empty
_devices = functools.lru_cache(None)(lambda index: torch.device("cuda", index))  # (an index costs torch.empty 2 us more)


def _output(t, name: str, dtype, device: int, shape):
    """(tensor, address) of an output: the caller's, checked, or a new one."""
    if t is None:
        t = _empty(shape, dtype=dtype, device=_devices(device))
        return t, t.data_ptr()
    return t, _shaped(t, name, dtype, device, shape)


_TYPES = {torch.float32: SSD_DTYPE_F32, torch.bfloat16: SSD_DTYPE_BF16}
_HERE = contextlib.nullcontext()
_Tensor = torch.Tensor
# What torch.cuda.current_stream, current_device and is_current_stream_capturing ask, without their objects and
# initialisation checks (a cache's tensors are on the device already): 1.5 us of a call that took 11.  A torch without
# these private names gets the public calls.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing


def _scope(device: int, stream):
    """The cache's device and the call's stream current, for allocations as for launches."""
    if stream is None:
        return _HERE if _current_device() == device else torch.cuda.device(device)
    if stream.device_index != device:
        raise ValueError(f"stream is on cuda:{stream.device_index}, expected cuda:{device}")
    return torch.cuda.stream(stream)


def _shaped(t, name: str, dtype, device: int, shape) -> int:
    """Address of a contiguous tensor of that type, device and shape."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == device and t.is_contiguous() and t.shape == shape:
        return t.data_ptr()
    _need(t, name, dtype, torch.device("cuda", device))  # says what is wrong
    raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _maybe(t, name: str, dtype, device: int, shape) -> Optional[int]:
    return None if t is None else _shaped(t, name, dtype, device, shape)


def _typed(t, name: str) -> int:
    code = _TYPES.get(t.dtype) if isinstance(t, _Tensor) else None
    if code is None:
        raise TypeError(f"{name} must be a bf16 or fp32 torch.Tensor, got {t.dtype if isinstance(t, _Tensor) else type(t).__name__}")
    return code


def _is_kv4(kv):
    if not isinstance(kv, KV4Cache):
        raise TypeError(f"kv must be a KV4Cache, got {type(kv).__name__}")


_STREAM_WS = {}  # (device, stream, name): buffer, aligned address, bytes from there
# Held from a call's look up of its workspace until its last launch: ctypes lets other threads run meanwhile, and two
# threads on one stream share a workspace, so their calls' launches must not fall between each other's.
_WS_LOCK = threading.RLock()


def _stream_ws(device: int, name: str, nbytes: int, workspace: Optional[Workspace], counters: bool = True):
    """Workspace of a call on the current stream: the caller's, or one kept for (device, stream), so that
    calls on different streams never share one; a call under stream capture without a workspace, or with one that an
    earlier call has not made large enough, takes a buffer of its graph's own memory, whose counters a node of the
    graph clears (calls without counters need none).  A caller's workspace that graphs were captured with must outlive them, and
    they run one after the other.  Under _WS_LOCK."""
    capturing = _capturing()
    if workspace is not None:
        at = torch.device("cuda", device)
        buf = workspace._bufs.get((str(at), name))
        if not capturing or (buf is not None and buf.numel() >= nbytes):
            if capturing and not any(b is buf for b in workspace._captured):
                workspace._captured.append(buf)
            return _ws(at, name, nbytes, workspace)
    if capturing:
        buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
        if counters:
            buf[:COUNTER_BYTES + 256].zero_()
        return Workspace.aligned(buf), nbytes
    key = (device, _raw_stream(device), name)
    kept = _STREAM_WS.get(key)
    if kept is None or kept[2] < nbytes:
        buf = torch.zeros(nbytes + 256, dtype=torch.uint8, device=device)
        kept = _STREAM_WS[key] = (buf, Workspace.aligned(buf), nbytes)
    return kept[1], kept[2]


def ssd_kv4_append(kv: KV4Cache, k_new: torch.Tensor, v_new: torch.Tensor, counts: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """Quantises rows k_new / v_new [B, n_new, h_kv, d] (bf16 or fp32) into positions seq_lens[b] + j of every
    request, j < counts[b] (int32 [B]; None: all n_new); kv.pool is modified in place, kv.seq_lens is not."""
    _is_kv4(kv)
    dev, B, h, d = kv._geometry
    dt = _typed(k_new, "k_new")
    n = k_new.shape[1] if k_new.dim() == 4 else -1
    if n < 0 or k_new.shape != (B, n, h, d):
        raise ValueError("k_new and v_new must both be [batch, n_new, h_kv, d]")
    pk = _shaped(k_new, "k_new", k_new.dtype, dev, (B, n, h, d))
    pv = _shaped(v_new, "v_new", k_new.dtype, dev, (B, n, h, d))
    pc = _maybe(counts, "counts", torch.int32, dev, (B,))
    if B == 0:  # (a tensor without elements has no address)
        return
    with _scope(dev, stream):
        _check(_lib().ssd_kv4_append(kv.ref(), pk, pv, dt, n, pc, kv.k_scale, kv.v_scale, _raw_stream(dev)))


def ssd_kv4_read(kv: KV4Cache, first: torch.Tensor, n: int, counts: Optional[torch.Tensor] = None, *, k=None, v=None,
                 dtype=torch.bfloat16, stream=None):
    """The values of the tokens first[b] + j, j < counts[b] (None: n), as k, v [B, n, h_kv, d] of `dtype` (bf16 or
    fp32; both exact); rows from counts[b] on are zeros."""
    _is_kv4(kv)
    dev, B, h, d = kv._geometry
    shape = (B, int(n), h, d)
    pf = _shaped(first, "first", torch.int32, dev, (B,))
    pc = _maybe(counts, "counts", torch.int32, dev, (B,))
    with _scope(dev, stream):
        if k is None:
            k = torch.empty(shape, dtype=dtype if v is None else v.dtype, device=dev)
        if v is None:
            v = torch.empty(shape, dtype=k.dtype, device=dev)
        dt = _typed(k, "k")
        pk = _shaped(k, "k", k.dtype, dev, shape)
        pv = _shaped(v, "v", k.dtype, dev, shape)
        if B:
            _check(_lib().ssd_kv4_read(kv.ref(), pf, pc, int(n), kv.k_scale, kv.v_scale, dt, pk, pv, _raw_stream(dev)))
    return k, v


def ssd_kv4_verify_attn(kv: KV4Cache, q: torch.Tensor, n_cand: int, scale: float, *, out=None, lse=None,
                        scores: Optional[torch.Tensor] = None, want_scores: bool = True, want_lse: bool = True,
                        out_dtype=torch.float32, workspace: Optional[Workspace] = None, stream=None) -> dict:
    """Verify attention over a 4-bit cache, with the tokens' criticality on request (n_cand = 1: plain
    decoding).  q [B, n_cand, h_q, d] bf16 or fp32; out fp32 or bf16 (`out_dtype` where it is not given)."""
    _is_kv4(kv)
    dev, B, h, d = kv._geometry
    qt = _typed(q, "q")
    h_q = q.shape[2] if q.dim() == 4 else -1
    shape = (B, n_cand, h_q, d)
    if q.shape != shape:
        raise ValueError("q must be [batch, n_cand, h_q, d]")
    pq = _shaped(q, "q", q.dtype, dev, shape)
    with _scope(dev, stream):
        if out is None:
            out = torch.empty(shape, dtype=out_dtype, device=dev)
        if lse is None and want_lse:
            lse = torch.empty(shape[:3], dtype=torch.float32, device=dev)
        if scores is None and want_scores:
            scores = torch.zeros((B, h, max(kv.max_seq_len, 1)), dtype=torch.float32, device=dev)
        ot = _typed(out, "out")
        po = _shaped(out, "out", out.dtype, dev, shape)
        pl = _maybe(lse, "lse", torch.float32, dev, shape[:3])
        stride = 0 if scores is None else scores.shape[-1] if scores.dim() else 0
        ps = _maybe(scores, "scores", torch.float32, dev, (B, h, stride))
        if B:
            L = _lib()
            need = kv._need.get((h_q, n_cand))
            if need is None:
                need = kv._need[h_q, n_cand] = L.ssd_kv4_verify_workspace_bytes(kv.ref(), h_q, n_cand)
            with _WS_LOCK:
                ws, avail = _stream_ws(dev, "kv4", need, workspace)
                _check(L.ssd_kv4_verify_attn(kv.ref(), pq, qt, h_q, n_cand, float(scale), kv.k_scale, kv.v_scale, po, ot, pl,
                                             ps, stride, ws, avail, _raw_stream(dev)))
    return {"out": out, "lse": lse, "scores": scores}


def ssd_kv4_draft_attn(kv: KV4Cache, q: torch.Tensor, idx: torch.Tensor, cnt: torch.Tensor, scale: float, *, out=None,
                       lse=None, want_lse: bool = True, out_dtype=torch.float32,
                       workspace: Optional[Workspace] = None, stream=None) -> dict:
    """Single-query attention over the selected tokens of a 4-bit cache.  q [B, h_q, d] bf16 or fp32;
    idx [B, h_kv, k_max] and cnt [B, h_kv] int32; out fp32 or bf16 (`out_dtype` where it is not given)."""
    _is_kv4(kv)
    dev, B, h, d = kv._geometry
    qt = _typed(q, "q")
    h_q = q.shape[1] if q.dim() == 3 else -1
    if q.shape != (B, h_q, d):
        raise ValueError("q must be [batch, h_q, d]")
    pq = _shaped(q, "q", q.dtype, dev, (B, h_q, d))
    if not isinstance(idx, torch.Tensor) or idx.dim() != 3:
        raise ValueError("idx must be [batch, h_kv, k_max]")
    k_max = idx.shape[2]
    pi = _shaped(idx, "idx", torch.int32, dev, (B, h, k_max))
    pc = _shaped(cnt, "cnt", torch.int32, dev, (B, h))
    with _scope(dev, stream):
        if out is None:
            out = torch.empty((B, h_q, d), dtype=out_dtype, device=dev)
        if lse is None and want_lse:
            lse = torch.empty((B, h_q), dtype=torch.float32, device=dev)
        ot = _typed(out, "out")
        po = _shaped(out, "out", out.dtype, dev, (B, h_q, d))
        pl = _maybe(lse, "lse", torch.float32, dev, (B, h_q))
        if B:
            L = _lib()
            need = kv._need.get((h_q, -1, k_max))
            if need is None:
                need = kv._need[h_q, -1, k_max] = L.ssd_kv4_draft_workspace_bytes(kv.ref(), h_q, k_max)
            with _WS_LOCK:
                ws, avail = _stream_ws(dev, "kv4", need, workspace)
                _check(L.ssd_kv4_draft_attn(kv.ref(), pq, qt, h_q, pi, k_max, pc, float(scale), kv.k_scale, kv.v_scale, po, ot,
                                            pl, ws, avail, _raw_stream(dev)))
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------------------------
# Pages of a cache: sharing, taking, giving back, compacting.
# ------------------------------------------------------------------------------------------------


@dataclass
class PagePool:
    """Reference counts of a pool's pages: refs int32 [num_pages], how many page-table entries hold each page
    (0 = free)."""
    refs: torch.Tensor

    def __post_init__(self):
        _need(self.refs, "refs", torch.int32)
        if self.refs.dim() != 1:
            raise ValueError("refs must be [num_pages]")

    @classmethod
    def from_table(cls, page_table: torch.Tensor, num_pages: int) -> "PagePool":
        """The counts of the pages a page table holds (entries >= 0, all of them below num_pages)."""
        held = page_table.reshape(-1)
        held = held[held >= 0].to(torch.int64)
        if held.numel() and int(held.max()) >= num_pages:
            raise ValueError(f"page_table names page {int(held.max())} of a pool of {num_pages} pages")
        refs = torch.zeros((num_pages,), dtype=torch.int32, device=page_table.device)
        return cls(refs.scatter_add_(0, held, torch.ones_like(held, dtype=torch.int32)))


def _pages_of(kv, pages: PagePool) -> int:
    if not isinstance(kv, (KVCache, KV4Cache)):
        raise TypeError(f"kv must be a KVCache or a KV4Cache, got {type(kv).__name__}")
    if not isinstance(pages, PagePool):
        raise TypeError(f"pages must be a PagePool, got {type(pages).__name__}")
    return _shaped(pages.refs, "pages.refs", torch.int32, kv._geometry[0], (kv._struct.num_pages,))


def _count(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 1:
        raise ValueError(f"{name} must be [n]")
    return t.shape[0]


def ssd_kv_fork(kv, pages: PagePool, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """Row dst[i] (empty before) shares the pages of row src[i] and takes its length; src, dst int32 [n].
    kv.page_table, kv.seq_lens and pages.refs are modified in place; no K / V moves."""
    refs = _pages_of(kv, pages)
    dev = kv._geometry[0]
    n = _count(src, "src")
    ps = _shaped(src, "src", torch.int32, dev, (n,))
    pd = _shaped(dst, "dst", torch.int32, dev, (n,))
    if n == 0:
        return
    with _scope(dev, stream):
        _check(_lib().ssd_kv_fork(kv.ref(), refs, ps, pd, n, _raw_stream(dev)))


def ssd_kv_reserve(kv, pages: PagePool, counts: torch.Tensor, *, workspace: Optional[Workspace] = None,
                   stream=None) -> None:
    """Pages of its own for the next counts[b] tokens of every request (int32 [B]); what a request shares there is
    copied.  All or nothing: with too few free pages the status reports FAULT_NOPAGE and nothing changes."""
    refs = _pages_of(kv, pages)
    dev, B = kv._geometry[:2]
    pc = _shaped(counts, "counts", torch.int32, dev, (B,))
    if B == 0:
        return
    with _scope(dev, stream):
        L = _lib()
        need = L.ssd_kv_reserve_workspace_bytes(kv.ref())
        with _WS_LOCK:
            ws, avail = _stream_ws(dev, "pages", need, workspace)
            _check(L.ssd_kv_reserve(kv.ref(), refs, pc, ws, avail, _raw_stream(dev)))


def ssd_kv_release(kv, pages: PagePool, keep: torch.Tensor, stream=None) -> None:
    """Row b gives back the pages behind its first keep[b] tokens (int32 [B]; 0: all, negative: none) and its
    length becomes min(length, keep[b])."""
    refs = _pages_of(kv, pages)
    dev, B = kv._geometry[:2]
    pk = _shaped(keep, "keep", torch.int32, dev, (B,))
    if B == 0:
        return
    with _scope(dev, stream):
        _check(_lib().ssd_kv_release(kv.ref(), refs, pk, _raw_stream(dev)))


def ssd_kv_compact(kv, to, src: torch.Tensor, dst: torch.Tensor, idx: torch.Tensor, cnt: torch.Tensor,
                   pages: Optional[PagePool] = None, stream=None) -> None:
    """The listed tokens idx [n, h_kv, k_max] (cnt [n, h_kv] of them, the same for every head) of row src[i] of `kv`
    go to positions 0 .. of row dst[i] of `to`, whose length becomes the count.  dst's pages are reserved
    beforehand; with `pages` (the PagePool of `to`) shared ones are left alone and reported, without it the caller
    answers for their being held by dst alone."""
    if not isinstance(kv, (KVCache, KV4Cache)) or type(to) is not type(kv):
        raise TypeError("kv and to must both be a KVCache or both a KV4Cache")
    dev, _, h, _ = kv._geometry
    refs = None if pages is None else _pages_of(to, pages)
    if to._geometry[0] != dev:
        raise ValueError(f"to is on {to.device}, expected {kv.device}")
    if isinstance(kv, KV4Cache) and (kv.k_scale, kv.v_scale) != (to.k_scale, to.v_scale):
        raise ValueError("the two caches differ in k_scale or v_scale")
    n = _count(src, "src")
    ps = _shaped(src, "src", torch.int32, dev, (n,))
    pd = _shaped(dst, "dst", torch.int32, dev, (n,))
    if not isinstance(idx, torch.Tensor) or idx.dim() != 3:
        raise ValueError("idx must be [n, h_kv, k_max]")
    k_max = idx.shape[2]
    pi = _shaped(idx, "idx", torch.int32, dev, (n, h, k_max))
    pc = _shaped(cnt, "cnt", torch.int32, dev, (n, h))
    if n == 0:
        return
    with _scope(dev, stream):
        _check(_lib().ssd_kv_compact(kv.ref(), to.ref(), refs, ps, pd, n, pi, k_max, pc, _raw_stream(dev)))


# ------------------------------------------------------------------------------------------------
# A step that drafts a tree of tokens: attention of a request's last tokens, scores, acceptance, commit.
# ------------------------------------------------------------------------------------------------


def _span_attn(kv, q, parents, counts, window, sink, scale, out, lse, want_lse, workspace, stream) -> dict:
    if not isinstance(kv, KVCache):
        raise TypeError(f"kv must be a KVCache, got {type(kv).__name__}")
    dev, B, h, d = kv._geometry
    if not isinstance(q, _Tensor) or q.dim() != 4:
        raise ValueError("q must be a torch.Tensor [batch, n, h_q, d]")
    n, h_q = q.shape[1], q.shape[2]
    shape = (B, n, h_q, d)
    dtype = kv.pool.dtype
    pq = _shaped(q, "q", dtype, dev, shape)
    pp = None if window is not None else _shaped(parents, "parents", torch.int32, dev, (B, n))
    pc = _maybe(counts, "counts", torch.int32, dev, (B,))
    with _scope(dev, stream):
        out, po = _output(out, "out", dtype, dev, shape)
        pl = None
        if lse is not None or want_lse:
            lse, pl = _output(lse, "lse", torch.float32, dev, shape[:3])
        if B:
            L = _lib()
            key = (h_q, n, window, sink)
            need = kv._need.get(key)
            if need is None:
                need = kv._need[key] = L.ssd_tree_workspace_bytes(kv.ref(), h_q, n) if window is None else \
                    L.ssd_window_workspace_bytes(kv.ref(), h_q, n, window, sink)
            with _WS_LOCK:
                ws, avail = _stream_ws(dev, "span", need, workspace, False)
                st = _raw_stream(dev)
                _check(L.ssd_tree_attn(kv.ref(), pq, h_q, n, pp, pc, scale, po, pl, ws, avail, st) if window is None else
                       L.ssd_window_attn(kv.ref(), pq, h_q, n, pc, window, sink, scale, po, pl, ws, avail, st))
    return {"out": out, "lse": lse}


def ssd_tree_attn(kv: KVCache, q: torch.Tensor, parents: torch.Tensor, scale: float, *, counts: Optional[torch.Tensor] = None,
                  out=None, lse=None, want_lse: bool = True, workspace: Optional[Workspace] = None, stream=None) -> dict:
    """Attention of a drafted tree over the paged cache: the nodes are the last counts[b] (int32 [B]; None: n) tokens of
    request b, and node i sees all tokens before the tree, its ancestors and itself.  q [B, n, h_q, d] and out have the
    cache's type; parents int32 [B, n], the earlier node that a node hangs on or -1.  Rows behind counts[b]: out 0,
    lse -inf."""
    return _span_attn(kv, q, parents, counts, None, 0, float(scale), out, lse, want_lse, workspace, stream)


def ssd_window_attn(kv: KVCache, q: torch.Tensor, window: int, sink: int, scale: float, *, counts: Optional[torch.Tensor] = None,
                    out=None, lse=None, want_lse: bool = True, workspace: Optional[Workspace] = None, stream=None) -> dict:
    """Attention of each request's last counts[b] (int32 [B]; None: n) tokens, a decoding step's one or a prompt's many, with
    a sliding window: position p sees the tokens t <= p with t > p - window or t < sink.  q [B, n, h_q, d] and out have the
    cache's type.  Rows behind counts[b]: out 0, lse -inf."""
    return _span_attn(kv, q, None, counts, _c_int(window, "window"), _c_int(sink, "sink"), float(scale), out, lse, want_lse, workspace, stream)


def ssd_token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *, rows: Optional[torch.Tensor] = None, top_k: int = 0,
                       logprob=None, lse=None, entropy=None, top_ids=None, top_logprobs=None, stream=None) -> dict:
    """Log probabilities of given tokens under rows of logits [N, V] (bf16 or fp32; rows may be strided), with every row's
    log-sum-exp and entropy and, for top_k > 0, its top_k largest logits' ids and log probabilities (descending, equal ones
    by index).  tokens int32: [N] or [N, m], each row's own, or with rows (int32 [M]) [M], token i looked up in row
    rows[i] (-1: a tree's root, which gets 0)."""
    dt = _typed(logits, "logits")
    if logits.dim() != 2 or not logits.is_cuda or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a CUDA tensor [rows, vocab] with its last dimension dense")
    N, V = _c_int(logits.shape[0], "rows"), _c_int(logits.shape[1], "vocab")
    dev = logits.get_device()
    M = 0
    pt = pr = None
    if tokens is not None:
        if not isinstance(tokens, _Tensor):
            raise TypeError("tokens must be a torch.Tensor")
        pt = _shaped(tokens, "tokens", torch.int32, dev, tokens.shape)
        M = _c_int(tokens.numel(), "tokens")
        if rows is not None:
            pr = _shaped(rows, "rows", torch.int32, dev, tokens.shape)
        elif tokens.dim() not in (1, 2) or tokens.shape[0] != N:
            raise ValueError("tokens must be [rows] or [rows, m]; give rows= for tokens of chosen rows")
    elif rows is not None or logprob is not None:
        raise ValueError("rows and logprob go with tokens")
    if top_k < 0 or top_k > V:
        raise ValueError(f"top_k {top_k} outside [0, {V}]")
    with _scope(dev, stream):
        f32, i32 = torch.float32, torch.int32
        pg = pi = pv = None
        if tokens is not None:
            logprob, pg = _output(logprob, "logprob", f32, dev, tokens.shape)
        lse, pl = _output(lse, "lse", f32, dev, (N,))
        entropy, pe = _output(entropy, "entropy", f32, dev, (N,))
        if top_k:
            top_ids, pi = _output(top_ids, "top_ids", i32, dev, (N, top_k))
            top_logprobs, pv = _output(top_logprobs, "top_logprobs", f32, dev, (N, top_k))
        if N or M:
            _check(_lib().ssd_token_logprobs(logits.data_ptr(), dt, logits.stride(0), N, V, pt, pr, M, pg, pl, pe, pi, pv, top_k,
                                             _raw_stream(dev)))
    return {"logprob": logprob, "lse": lse, "entropy": entropy, "top_ids": top_ids, "top_logprobs": top_logprobs}


def ssd_tree_accept(parents: torch.Tensor, tokens: Optional[torch.Tensor], target: torch.Tensor, *, counts: Optional[torch.Tensor] = None,
                    max_path: Optional[int] = None, logprob: Optional[torch.Tensor] = None,
                    entropy: Optional[torch.Tensor] = None, epsilon: float = 0.0, delta: float = 0.0, path=None, cnt=None,
                    next=None, advance=None, stream=None) -> dict:
    """The path of a drafted tree that stays.  parents, tokens, target int32 [B, n]: node 0 is the last step's token and
    stays; node c stays when its parent does and tokens[c] equals target[parent], or, with logprob and entropy (float
    [B, n]; tokens may then be None), when logprob[c] > min(ln epsilon, ln delta - entropy[parent]).  The deepest such node
    below max_path (None: n) gives path int32 [B, max_path] (-1 behind it), cnt, next = its target, and advance =
    cnt - counts for ``ssd_kv_advance``."""
    if not isinstance(parents, _Tensor) or parents.dim() != 2 or not parents.is_cuda:
        raise ValueError("parents must be a CUDA tensor [batch, n]")
    B, n = _c_int(parents.shape[0], "batch"), _c_int(parents.shape[1], "n")
    dev = parents.get_device()
    i32, f32 = torch.int32, torch.float32
    pp = _shaped(parents, "parents", i32, dev, (B, n))
    if tokens is None and logprob is None:
        raise ValueError("tokens or logprob must be given")
    pt = _maybe(tokens, "tokens", i32, dev, (B, n))
    pg = _shaped(target, "target", i32, dev, (B, n))
    pc = _maybe(counts, "counts", i32, dev, (B,))
    if (logprob is None) != (entropy is None):
        raise ValueError("logprob and entropy go together")
    pl = _maybe(logprob, "logprob", f32, dev, (B, n))
    pe = _maybe(entropy, "entropy", f32, dev, (B, n))
    m = n if max_path is None else _c_int(max_path, "max_path")
    if m < 1:
        raise ValueError(f"max_path {m} < 1")
    with _scope(dev, stream):
        path, ph = _output(path, "path", i32, dev, (B, m))
        cnt, pk = _output(cnt, "cnt", i32, dev, (B,))
        next, pn = _output(next, "next", i32, dev, (B,))
        advance, pa = _output(advance, "advance", i32, dev, (B,))
        if B:
            _check(_lib().ssd_tree_accept(pp, pt, pg, pl, pe, float(epsilon), float(delta), pc, B, n, m, ph, pk, pn, pa, _raw_stream(dev)))
    return {"path": path, "cnt": cnt, "next": next, "advance": advance}


def ssd_tree_commit(kv: KVCache, path: torch.Tensor, cnt: torch.Tensor, n: int, *, counts: Optional[torch.Tensor] = None, stream=None) -> None:
    """Moves the K and V rows of the nodes path[b, :cnt[b]] (int32 [B, max_path], ascending; int32 [B]) of each request's tree,
    its last counts[b] (int32 [B]; None: n) tokens, to the tree's first positions.  kv.pool is modified in place,
    kv.seq_lens is not: ``ssd_kv_advance`` it once every layer is done.  The tree's pages are the request's own."""
    if not isinstance(kv, KVCache):
        raise TypeError(f"kv must be a KVCache, got {type(kv).__name__}")
    dev, B = kv._geometry[:2]
    if not isinstance(path, _Tensor) or path.dim() != 2:
        raise ValueError("path must be a torch.Tensor [batch, max_path]")
    m = _c_int(path.shape[1], "max_path")
    pp = _shaped(path, "path", torch.int32, dev, (B, m))
    pk = _shaped(cnt, "cnt", torch.int32, dev, (B,))
    pc = _maybe(counts, "counts", torch.int32, dev, (B,))
    if B == 0:
        return
    with _scope(dev, stream):
        _check(_lib().ssd_tree_commit(kv.ref(), _c_int(n, "n"), pc, pp, m, pk, _raw_stream(dev)))
