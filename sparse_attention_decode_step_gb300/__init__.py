"""Thin Python binding of the CSA2 C ABI (include/csa2.h).

Argument marshalling only: tensors become device pointers, and every step of
the path runs in the CUDA library libcsa2.so.  There is no fallback: if the
library is missing or a call fails, an exception is raised.  PyTorch supplies
device memory and the current CUDA stream.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

import torch

from . import build as _build

FULL, REINDEX, REUSE = 0, 1, 2
D = 512
CNT_FP4_SATURATED, CNT_CAPACITY, CNT_BAD_INPUT, CNT_TIMEOUT = 0, 1, 2, 3
NUM_COUNTERS = 4

_lock = threading.Lock()
_lib = None

_STATUS = {0: "ok", -1: "invalid argument", -2: "pointer not 16-byte aligned",
           -3: "workspace or output too small", -4: "shape not supported", -5: "CUDA error"}

EXPORTS = ["csa2_quantize_append", "csa2_quantize_append_project", "csa2_index_full", "csa2_index_reindex", "csa2_topk",
           "csa2_pool_select", "csa2_sparse_attn", "csa2_layer_step", "csa2_index_workspace_size",
           "csa2_topk_workspace_size", "csa2_attn_workspace_size", "csa2_layer_workspace_size",
           "csa2_status_string", "csa2_launch_count", "csa2_topk_noalloc",
           "csa2_topk_noalloc_max_scratch", "csa2_cache_write", "csa2_cache_read",
           "csa2_dense_attn", "csa2_dense_workspace_size", "csa2_norm_rope", "csa2_chunk_attn",
           "csa2_attn_mass", "csa2_mass_workspace_size", "csa2_cache_evict", "csa2_evict_workspace_size"]


class CsaError(RuntimeError):
    pass


class _Cache(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("kidx", ctypes.c_void_p),
                ("kscale", ctypes.c_void_p), ("seq_base", ctypes.c_void_p),
                ("seq_len", ctypes.c_void_p), ("cap", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("d_idx", ctypes.c_int32), ("m", ctypes.c_int32)]


class _Queries(ctypes.Structure):
    _fields_ = [("q_seq", ctypes.c_void_p), ("q_pos", ctypes.c_void_p), ("nq", ctypes.c_int32),
                ("group", ctypes.c_int32)]


class _Groups(ctypes.Structure):
    _fields_ = [("seq", ctypes.c_void_p), ("off", ctypes.c_void_p), ("len", ctypes.c_void_p),
                ("ng", ctypes.c_int32), ("nq", ctypes.c_int32)]


class _Pages(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("ld", ctypes.c_int64), ("page", ctypes.c_int32)]


class _LayerArgs(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("cache", ctypes.c_void_p), ("queries", ctypes.c_void_p),
                ("q_idx", ctypes.c_void_p), ("w", ctypes.c_void_p), ("h_idx", ctypes.c_int32),
                ("max_n", ctypes.c_int64), ("k", ctypes.c_int32), ("build_pool", ctypes.c_int32),
                ("pool_blocks", ctypes.c_int32), ("pool_blk", ctypes.c_void_p),
                ("pool_n", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("cnt", ctypes.c_void_p),
                ("q", ctypes.c_void_p), ("H", ctypes.c_int32), ("win", ctypes.c_void_p),
                ("wcap", ctypes.c_int32), ("win_start", ctypes.c_void_p),
                ("n_win", ctypes.c_int32), ("sm_scale", ctypes.c_float), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t), ("counters", ctypes.c_void_p)]


def library_path() -> str:
    return _build.LIB_PATH


def lib() -> ctypes.CDLL:
    """Loads libcsa2.so, building it with nvcc first if it is missing or stale."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            if not os.path.exists(path):
                raise CsaError(f"CUDA library not found at {path}")
            L = ctypes.CDLL(path)
            vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
            sig = {
                "csa2_quantize_append": [vp, vp, vp, vp, i32, vp, vp],
                "csa2_quantize_append_project": [vp, vp, vp, vp, i32, vp, vp],
                "csa2_index_full": [vp, vp, vp, vp, i32, i64, vp, i64, vp, i64, vp, vp, sz, vp, vp],
                "csa2_index_reindex": [vp, vp, vp, vp, i32, vp, vp, i32, vp, i64, vp, vp, sz, vp,
                                       vp],
                "csa2_topk": [vp, i64, vp, vp, i32, i32, i64, i32, vp, i64, vp, vp, sz, vp],
                "csa2_pool_select": [vp, i64, vp, i32, i64, i32, vp, vp, vp, sz, vp],
                "csa2_sparse_attn": [vp, vp, vp, i64, vp, i32, vp, i32, vp, i32, vp, i32,
                                     ctypes.c_float, vp, vp, vp, sz, vp, vp],
                "csa2_layer_step": [vp, vp],
                "csa2_cache_write": [vp, vp, i64, vp, i32, i64, vp, i64, vp, vp],
                "csa2_cache_read": [vp, vp, i64, vp, i32, i64, vp, i64, vp, vp],
                "csa2_dense_attn": [vp, vp, i64, vp, i32, i32, ctypes.c_float, vp, vp, vp, i32, vp,
                                    vp, sz, vp, vp],
                "csa2_norm_rope": [vp, i32, i64, i64, i32, vp, ctypes.c_float, vp, vp, i32, i32, vp, i32, i64, vp],
                "csa2_chunk_attn": [vp, vp, vp, vp, i64, vp, i32, i32, ctypes.c_float, vp, vp, vp, i32, vp,
                                    vp, sz, vp, vp],
                "csa2_attn_mass": [vp, vp, vp, vp, i64, vp, i32, i32, ctypes.c_float, vp, vp, ctypes.c_float, vp, i64,
                                   vp, sz, vp, vp],
                "csa2_cache_evict": [vp, vp, vp, vp, vp, i32, vp, i64, i64, i32, i32, i32, vp, i64, vp, i64,
                                     vp, sz, vp, vp],
            }
            for name, args in sig.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = ctypes.c_int
            L.csa2_index_workspace_size.argtypes = [i32, i32, i32, i32]
            L.csa2_index_workspace_size.restype = sz
            L.csa2_topk_workspace_size.argtypes = [i32, i64]
            L.csa2_topk_workspace_size.restype = sz
            L.csa2_attn_workspace_size.argtypes = [i32, i32, i32, i32]
            L.csa2_attn_workspace_size.restype = sz
            L.csa2_layer_workspace_size.argtypes = [vp]
            L.csa2_layer_workspace_size.restype = sz
            L.csa2_dense_workspace_size.argtypes = [i32, i32, i32, i64]
            L.csa2_dense_workspace_size.restype = sz
            L.csa2_mass_workspace_size.argtypes = [i32, i32, i32, i32, i64]
            L.csa2_mass_workspace_size.restype = sz
            L.csa2_evict_workspace_size.argtypes = [i32, i64]
            L.csa2_evict_workspace_size.restype = sz
            L.csa2_status_string.argtypes = [ctypes.c_int]
            L.csa2_status_string.restype = ctypes.c_char_p
            L.csa2_launch_count.argtypes = []
            L.csa2_launch_count.restype = ctypes.c_uint64
            _lib = L
    return _lib


def _check(status: int, what: str):
    if status != 0:
        raise CsaError(f"{what}: {_STATUS.get(status, status)}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise CsaError("tensor is not on a CUDA device")
    if not t.is_contiguous():
        raise CsaError("tensor is not contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def launch_count() -> int:
    return int(lib().csa2_launch_count())


# ---------------------------------------------------------------- state
class Cache:
    """An FP4 main-KV cache with FP8 indexer keys, in device memory.

    `lengths_cap[b]` is the capacity of sequence b (entries); rows are laid
    out back to back with each sequence starting on a multiple of 8."""

    def __init__(self, lengths_cap, d_idx: int, m: int, device="cuda"):
        caps = [int(-(-int(c) // 8) * 8) for c in lengths_cap]
        base = [0]
        for c in caps:
            base.append(base[-1] + c)
        self.batch = len(caps)
        self.cap = max(8, base[-1])
        self.d_idx = d_idx
        self.m = m
        dev = torch.device(device)
        self.codes = torch.zeros(self.cap, 256, dtype=torch.uint8, device=dev)
        self.scales = torch.zeros(self.cap, 32, dtype=torch.uint8, device=dev)
        self.kidx = torch.zeros(self.cap, d_idx, dtype=torch.uint8, device=dev)
        self.kscale = torch.zeros(self.cap, dtype=torch.float32, device=dev)
        self.seq_base = torch.tensor(base, dtype=torch.int64, device=dev)
        self.seq_len = torch.zeros(self.batch, dtype=torch.int32, device=dev)
        self.base_host = base

    @classmethod
    def over(cls, codes, scales, kidx, kscale, seq_base, seq_len, m: int) -> "Cache":
        """A cache over tensors that the caller already holds (nothing is copied):
        codes [cap][256], scales [cap][32], kidx [cap][d_idx] uint8, kscale [cap]
        fp32, seq_base [batch + 1] int64, seq_len [batch] int32, cap a multiple of 8.
        kidx and kscale may be None for a cache that is only attended, seq_base for
        one whose sequences lie in pages (Pages)."""
        c = cls.__new__(cls)
        c.cap, c.batch, c.d_idx = (_ext or _load_ext()).check_cache(codes, scales, kidx, kscale, seq_base, seq_len)
        c.m = m
        c.codes, c.scales, c.kidx, c.kscale = codes, scales, kidx, kscale
        c.seq_base, c.seq_len, c.base_host = seq_base, seq_len, None
        return c

    def struct(self, seq=None) -> _Cache:
        """The C struct; with seq = b, a one-sequence view of sequence b."""
        keys = (None, None) if self.kidx is None else (self.kidx.data_ptr(), self.kscale.data_ptr())
        if self.seq_base is None:
            raise CsaError("the cache has no seq_base: its sequences lie in pages")
        if seq is None:
            return _Cache(self.codes.data_ptr(), self.scales.data_ptr(), *keys,
                          self.seq_base.data_ptr(), self.seq_len.data_ptr(),
                          self.cap, self.batch, self.d_idx, self.m)
        return _Cache(self.codes.data_ptr(), self.scales.data_ptr(), *keys,
                      self.seq_base.data_ptr() + 8 * int(seq),
                      self.seq_len.data_ptr() + 4 * int(seq), self.cap, 1, self.d_idx, self.m)


class Queries:
    def __init__(self, q_seq, q_pos, group: int = 1, device="cuda"):
        self.q_seq = torch.as_tensor(q_seq, dtype=torch.int32).to(device).contiguous()
        self.q_pos = torch.as_tensor(q_pos, dtype=torch.int32).to(device).contiguous()
        self.nq = int(self.q_seq.numel())
        self.group = group

    def struct(self) -> _Queries:
        return _Queries(self.q_seq.data_ptr(), self.q_pos.data_ptr(), self.nq, self.group)


class Groups:
    """Query groups of dense_attn: group g is the queries off[g] .. off[g+1]-1 and
    attends to the first length[g] entries (None: all) of sequence seq[g]."""

    def __init__(self, seq, off, length=None, device="cuda"):
        def dev(t):
            if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.int32 and t.is_contiguous():
                return t
            return torch.as_tensor(t, dtype=torch.int32).to(device).contiguous()
        self.seq, self.off = dev(seq), dev(off)
        self.length = None if length is None else dev(length)
        self.ng = self.seq.numel()
        if self.off.numel() != self.ng + 1 or (length is not None and self.length.numel() != self.ng):
            raise CsaError("groups need seq [ng], off [ng + 1] and length [ng]")


class Pages:
    """Where the sequences of a cache lie that are given pages as they grow: entry j of
    sequence b is row table[b][j // page] * page + j % page.  table: int32 [batch][pages]
    (what lies behind a sequence's pages may be anything), page: a power of two from 16 on."""

    def __init__(self, table, page: int, device="cuda"):
        if not (isinstance(table, torch.Tensor) and table.dtype == torch.int32 and table.is_contiguous() and
                (table.is_cuda or torch.device(device).type == "cpu")):
            table = torch.as_tensor(table, dtype=torch.int32).to(device).contiguous()
        page = int(page)
        if table.dim() != 2 or page < 16 or page & (page - 1):
            raise CsaError("pages need a table [sequences][pages] and a power of two of entries per page, 16 or more")
        self.table, self.page = table, page

    def rows(self, seq, entry):
        """Cache rows of entries `entry` of sequences `seq` (integer tensors), for cache_write and cache_read."""
        entry = entry.long()
        return self.table[seq.long(), entry // self.page].long() * self.page + entry % self.page


def new_counters(device="cuda"):
    return torch.zeros(NUM_COUNTERS, dtype=torch.int32, device=device)


def workspace(nbytes: int, device="cuda"):
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- entry points
def quantize_append(cache: Cache, C, Z, key, counters=None, seq=None):
    """Appends C.shape[1] tokens to every sequence (or only to sequence `seq`)."""
    n_tok = int(C.shape[1])
    cs = cache.struct(seq)
    _check(lib().csa2_quantize_append(ctypes.byref(cs), _ptr(C), _ptr(Z), _ptr(key), n_tok,
                                      _ptr(counters), _stream()), "csa2_quantize_append")


def quantize_append_project(cache: Cache, C, Z, w_ik, counters=None, seq=None):
    """Appends C.shape[1] tokens to every sequence (or only to sequence `seq`),
    each entry's indexer key projected from the stored entry by w_ik, a bf16
    tensor [512][d_idx]."""
    if w_ik.dtype != torch.bfloat16 or tuple(w_ik.shape) != (512, cache.d_idx):
        raise CsaError(f"w_ik must be bf16 [512][{cache.d_idx}], got {w_ik.dtype} {tuple(w_ik.shape)}")
    n_tok = int(C.shape[1])
    cs = cache.struct(seq)
    _check(lib().csa2_quantize_append_project(ctypes.byref(cs), _ptr(C), _ptr(Z),
                                              _ptr(w_ik.contiguous()), n_tok, _ptr(counters),
                                              _stream()),
           "csa2_quantize_append_project")


def index_workspace_size(nq, group, h_idx, d_idx) -> int:
    return int(lib().csa2_index_workspace_size(nq, group, h_idx, d_idx))


def topk_workspace_size(nq, max_n) -> int:
    return int(lib().csa2_topk_workspace_size(nq, max_n))


def attn_workspace_size(nq, H, k_max, n_win) -> int:
    return int(lib().csa2_attn_workspace_size(nq, H, k_max, n_win))


def index_full(cache: Cache, qs: Queries, q_idx, w, max_n, scores, blockmax=None, n_valid=None,
               ws=None, counters=None):
    h_idx = int(q_idx.shape[1])
    if ws is None:
        ws = workspace(index_workspace_size(qs.nq, qs.group, h_idx, cache.d_idx), q_idx.device)
    cs, qq = cache.struct(), qs.struct()
    _check(lib().csa2_index_full(ctypes.byref(cs), ctypes.byref(qq), _ptr(q_idx), _ptr(w), h_idx,
                                 int(max_n), _ptr(scores), int(scores.shape[1]), _ptr(blockmax),
                                 int(blockmax.shape[1]) if blockmax is not None else 0,
                                 _ptr(n_valid), _ptr(ws), ws.numel(), _ptr(counters), _stream()),
           "csa2_index_full")


def index_reindex(cache: Cache, qs: Queries, q_idx, w, pool_blk, pool_n, scores, n_valid=None,
                  ws=None, counters=None):
    h_idx = int(q_idx.shape[1])
    if ws is None:
        ws = workspace(index_workspace_size(qs.nq, 1, h_idx, cache.d_idx), q_idx.device)
    cs, qq = cache.struct(), qs.struct()
    _check(lib().csa2_index_reindex(ctypes.byref(cs), ctypes.byref(qq), _ptr(q_idx), _ptr(w),
                                    h_idx, _ptr(pool_blk), _ptr(pool_n), int(pool_blk.shape[1]),
                                    _ptr(scores), int(scores.shape[1]), _ptr(n_valid), _ptr(ws),
                                    ws.numel(), _ptr(counters), _stream()), "csa2_index_reindex")


def topk(scores, n_valid, k, idx_out, cnt_out, max_n=None, pool_blk=None, ws=None):
    nq = int(scores.shape[0])
    max_n = int(scores.shape[1] if max_n is None else max_n)
    if ws is None:
        ws = workspace(topk_workspace_size(nq, max_n), scores.device)
    _check(lib().csa2_topk(_ptr(scores), int(scores.shape[1]), _ptr(n_valid), _ptr(pool_blk),
                           int(pool_blk.shape[1]) if pool_blk is not None else 0, nq, max_n,
                           int(k), _ptr(idx_out), int(idx_out.shape[1]), _ptr(cnt_out), _ptr(ws),
                           ws.numel(), _stream()), "csa2_topk")


def pool_select(blockmax, n_valid, max_n, pool_blk, pool_n, ws=None):
    nq = int(blockmax.shape[0])
    if ws is None:
        ws = workspace(topk_workspace_size(nq, (int(max_n) + 7) // 8), blockmax.device)
    _check(lib().csa2_pool_select(_ptr(blockmax), int(blockmax.shape[1]), _ptr(n_valid), nq,
                                  int(max_n), int(pool_blk.shape[1]), _ptr(pool_blk),
                                  _ptr(pool_n), _ptr(ws), ws.numel(), _stream()),
           "csa2_pool_select")


def sparse_attn(cache: Cache, qs: Queries, idx, cnt, q, win, n_win, out, lse=None, win_start=None,
                sm_scale=1.0, k_max=None, ws=None, counters=None):
    H = int(q.shape[1])
    k_max = int(idx.shape[1] if (k_max is None and idx is not None) else (k_max or 0))
    wcap = int(win.shape[1]) if win is not None else 0
    if ws is None:
        ws = workspace(attn_workspace_size(qs.nq, H, k_max, n_win), q.device)
    cs, qq = cache.struct(), qs.struct()
    _check(lib().csa2_sparse_attn(ctypes.byref(cs), ctypes.byref(qq), _ptr(idx),
                                  int(idx.shape[1]) if idx is not None else 0, _ptr(cnt), k_max,
                                  _ptr(q), H, _ptr(win), wcap, _ptr(win_start), int(n_win),
                                  float(sm_scale), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                  _ptr(counters), _stream()), "csa2_sparse_attn")


# The calls below are short on the GPU, so their tensors are checked and taken
# apart in compiled code (csrc/csa2_torch.cpp) instead of here.
_ext = None


def _load_ext():
    """Loads csa2_torch.so, building it with g++ first if it is missing, stale or of
    another PyTorch.  Only Cache.over and the calls below need it."""
    global _ext
    lib()
    with _lock:
        if _ext is None:
            loader = importlib.machinery.ExtensionFileLoader("csa2_torch", _build.build_ext())
            mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("csa2_torch", loader))
            loader.exec_module(mod)
            mod.set_errors(CsaError, torch.OutOfMemoryError)
            _ext = mod
    return _ext


def cache_write(cache: Cache, rows, x, key=None, counters=None):
    """Quantises x [n][512] (fp32, bf16 or f16; rows 512 elements or more and a multiple
    of 16 bytes apart) into the cache rows rows [n] (int64, distinct; negative: skipped),
    and key [n][d_idx] (x's type, its rows likewise) into their indexer keys if it is given."""
    (_ext or _load_ext()).cache_write(cache, rows, x, key, counters)


def cache_read(cache: Cache, rows, x, key=None, counters=None):
    """Reads the cache rows rows [n] (int64; negative: skipped) into x [n][512] (fp32,
    bf16 or f16: exact) and, if given, their indexer keys into key [n][d_idx] fp32; rows
    of x and key lie apart as in cache_write."""
    (_ext or _load_ext()).cache_read(cache, rows, x, key, counters)


def dense_workspace_size(ng, nq, H, max_n) -> int:
    return int(lib().csa2_dense_workspace_size(ng, nq, H, max_n))


def dense_attn(cache: Cache, groups: Groups, q, out, lse=None, *, prev=None, sm_scale=1.0,
               max_n=None, ws=None, counters=None):
    """Attention of each group's queries q [nq][H][512] (bf16 or f16) over all the
    entries of the group's sequence, into out [nq][H][512] (fp32, bf16 or f16) and
    lse [nq][H]; prev = (out, lse) of an earlier partial result (fp32) is merged in.
    max_n bounds the entries of any group (default: the cache's rows).  q, out, lse and
    prev are contiguous.  Every entry counts: this is not the selection of sparse_attn."""
    try:
        seq, off, length = groups.seq, groups.off, groups.length
        po, pl = prev if prev is not None else (None, None)
    except (AttributeError, TypeError, ValueError) as e:
        raise CsaError("dense_attn: groups must be Groups, prev a pair (out, lse)") from e
    (_ext or _load_ext()).dense_attn(cache, seq, off, length, q, out, lse, po, pl, sm_scale, max_n, ws, counters)


def norm_rope(x, out, *, weight=None, eps=1e-6, pos=None, inv_freq=None, halves=False):
    """RMS norm of every row of x [n][H][512] or [n][512] (fp32, bf16 or f16; a token's heads
    side by side, tokens any multiple of 16 bytes apart), times weight [512] (fp32), and the
    rotation of its last 2 * len(inv_freq) channels (a multiple of 16) by the angles
    pos[i] * inv_freq (int32 [n], fp32), into out, which may be x.  Pairs are neighbours, or
    with halves=True half the rotated channels apart."""
    (_ext or _load_ext()).norm_rope(x, out, weight, eps, pos, inv_freq, halves)


def _of_groups(groups, pages):
    try:
        table, page = (None, 0) if pages is None else (pages.table, pages.page)
        return groups.seq, groups.off, groups.length, table, page
    except AttributeError as e:
        raise CsaError("groups must be Groups, pages Pages") from e


def chunk_attn(cache: Cache, groups: Groups, q, out, lse=None, *, pos=None, pages=None, prev=None,
               sm_scale=1.0, max_n=None, ws=None, counters=None):
    """Attention of chunks of new tokens: like dense_attn, but group g's queries are consecutive
    tokens of its sequence from token position pos[g] (int32 [groups]) on, and each sees the
    entries up to its own, (position + 1) // m of them; their entries are in the cache already.
    pos=None: all see everything.  pages: a Pages, if the sequences lie in pages."""
    seq, off, length, table, page = _of_groups(groups, pages)
    try:
        po, pl = prev if prev is not None else (None, None)
    except (TypeError, ValueError) as e:
        raise CsaError("chunk_attn: prev must be a pair (out, lse)") from e
    (_ext or _load_ext()).chunk_attn(cache, seq, off, length, pos, table, page, q, out, lse, po, pl, sm_scale, max_n, ws,
                                     counters)


def mass_workspace_size(batch, ng, nq, H, max_n) -> int:
    return int(lib().csa2_mass_workspace_size(batch, ng, nq, H, max_n))


def attn_mass(cache: Cache, groups: Groups, q, lse, mass, *, pos=None, pages=None, prev=None, decay=1.0,
              sm_scale=1.0, max_n=None, ws=None, counters=None):
    """How much weight the queries of each group gave to each entry of its sequence, with the
    log sums lse [nq][H] that the attention left: mass[b][j] = decay * prev[b][j] + the sum over
    queries and heads (mass, prev fp32 [sequences][entries]; prev may be mass, None: nothing
    before).  groups, pos and pages as in chunk_attn; a sequence is in one group at most."""
    seq, off, length, table, page = _of_groups(groups, pages)
    (_ext or _load_ext()).attn_mass(cache, seq, off, length, pos, table, page, q, lse, prev, decay, mass, sm_scale, max_n, ws,
                                    counters)


def evict_workspace_size(ns, max_n) -> int:
    return int(lib().csa2_evict_workspace_size(ns, max_n))


def cache_evict(cache: Cache, to: Cache, mass, keep, kept, mass_out=None, *, first=0, last=0, seq=None, pages=None,
                to_pages=None, max_n=None, ws=None, counters=None):
    """Cuts sequences (seq: int32 [ns]; None: all) to `keep` entries: the first `first`, the last
    `last`, and the rest by mass [sequences][entries] (ties to the lower entry).  They are copied
    in order to the entries 0, 1, .. of the same sequence of `to`, whose seq_len is set: the
    same tensors with other pages (to_pages), or another cache.  kept int32 [ns][keep] receives
    the old entry numbers, mass_out [sequences][keep] their mass.  max_n bounds the entries of
    any sequence (default: mass's width)."""
    def of(p):
        if p is None:
            return None, 0
        try:
            return p.table, p.page
        except AttributeError as e:
            raise CsaError("cache_evict: pages and to_pages must be Pages") from e
    (_ext or _load_ext()).cache_evict(cache, to, mass, keep, kept, mass_out, first, last, seq, *of(pages), *of(to_pages), max_n,
                                      ws, counters)


class Layer:
    """Arguments of one csa2_layer_step call; keeps the ctypes structures alive."""

    def __init__(self, mode, cache: Cache, qs: Queries, *, k, q, win, n_win, out, idx, cnt,
                 q_idx=None, w=None, max_n=0, build_pool=False, pool_blocks=2048, pool_blk=None,
                 pool_n=None, lse=None, win_start=None, sm_scale=1.0, counters=None, ws=None):
        self._cs = cache.struct()
        self._qs = qs.struct()
        self._keep = [q_idx, w, pool_blk, pool_n, idx, cnt, q, win, win_start, out, lse, counters]
        a = _LayerArgs()
        a.mode = int(mode)
        a.cache = ctypes.addressof(self._cs)
        a.queries = ctypes.addressof(self._qs)
        a.q_idx = q_idx.data_ptr() if q_idx is not None else None
        a.w = w.data_ptr() if w is not None else None
        a.h_idx = int(q_idx.shape[1]) if q_idx is not None else 0
        a.max_n = int(max_n)
        a.k = int(k)
        a.build_pool = int(bool(build_pool))
        a.pool_blocks = int(pool_blocks)
        a.pool_blk = pool_blk.data_ptr() if pool_blk is not None else None
        a.pool_n = pool_n.data_ptr() if pool_n is not None else None
        a.idx = idx.data_ptr()
        a.cnt = cnt.data_ptr()
        a.q = q.data_ptr()
        a.H = int(q.shape[1])
        a.win = win.data_ptr() if win is not None else None
        a.wcap = int(win.shape[1]) if win is not None else 0
        a.win_start = win_start.data_ptr() if win_start is not None else None
        a.n_win = int(n_win)
        a.sm_scale = float(sm_scale)
        a.out = out.data_ptr()
        a.lse = lse.data_ptr() if lse is not None else None
        a.counters = counters.data_ptr() if counters is not None else None
        self.args = a
        need = int(lib().csa2_layer_workspace_size(ctypes.byref(a)))
        if ws is None or ws.numel() < need:
            ws = workspace(need, q.device)
        self.ws = ws
        a.workspace = ws.data_ptr()
        a.ws_bytes = ws.numel()

    def __call__(self):
        _check(lib().csa2_layer_step(ctypes.byref(self.args), _stream()), "csa2_layer_step")
