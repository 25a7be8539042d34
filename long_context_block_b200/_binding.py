"""Thin ctypes binding over libmisa_b200.so (argument marshalling only).

Every function here has the name of the C entry point it calls (include/misa.h),
takes torch CUDA tensors, allocates the outputs and the workspace through torch,
and passes raw device pointers plus torch's current CUDA stream.  All computation
happens in the library's kernels; there is no CPU path.  A missing library raises
at import time.
"""

from __future__ import annotations

import array
import ctypes
import functools
import os
import re
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmisa_b200.so")
INCLUDE_DIR = os.path.join(os.path.dirname(_PKG), "include")
HEADER_PATH = os.path.join(INCLUDE_DIR, "misa.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python long_context_block_b200/build.py` "
        "(or __graft_entry__.build()); this package has no fallback path")

_lib = ctypes.CDLL(LIB_PATH)

_c_int, _c_i64, _c_sz, _p = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p

_SIGS = {
    "misa_workspace_size": (_c_sz, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_i64, _c_int,
                                    _c_int, _c_int, _c_int]),
    "misa_pool_keys": (_c_int, [_p, _c_int, _c_i64, _c_int, _c_int, _p, _p]),
    "misa_pool_keys_range": (_c_int, [_p, _c_int, _c_i64, _c_int, _c_int, _c_i64, _c_i64, _p,
                                      _p]),
    "misa_route_heads": (_c_int, [_p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int, _c_i64,
                                  _c_int, _c_int, _p, _p, _p, _c_sz, _p]),
    "misa_score_topk": (_c_int, [_p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int, _c_i64,
                                 _c_int, _c_int, _p, _p, _p, _p, _c_sz, _p]),
    "dsa_score_topk": (_c_int, [_p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int, _c_i64, _c_int,
                                _p, _p, _p, _p, _c_sz, _p]),
    "misa_dagger_rerank": (_c_int, [_p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int, _c_i64,
                                    _c_int, _c_int, _p, _p, _p, _c_sz, _p]),
    "misa_score_rows": (_c_int, [_p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int, _c_i64,
                                 _c_int, _p, _p, _c_sz, _p]),
    "misa_score_topk_noalloc": (_c_int, [_p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int,
                                         _c_i64, _c_int, _c_int, _p, _p, _p, _p]),
    "hisa_block_filter_topk": (_c_int, [_p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int,
                                        _c_i64, _c_int, _c_int, _c_int, _p, _p, _p, _p, _c_sz,
                                        _p]),
    "misa_paged_attention_workspace_size": (_c_sz, [_c_int] * 8),
    "misa_paged_attention": (_c_int, [_p] * 6 + [_c_int] * 10 + [ctypes.c_float] + [_p] * 4
                             + [_c_sz, _p]),
    "misa_testing_paged_attention_wait_expiry": (
        _c_int, [_p] * 6 + [_c_int] * 10 + [ctypes.c_float] + [_p] * 4
        + [_c_sz, ctypes.c_longlong, _c_int, _p]),
    "misa_paged_append": (_c_int, [_p] * 4 + [_c_int] * 8 + [_p] * 4),
    "misa_pages_workspace_size": (_c_sz, [_c_int] * 4),
    "misa_pages_resize": (_c_int, [_p] * 4 + [_c_int] * 4 + [_p, _p, _c_int] + [_p] * 4
                          + [_c_sz, _p]),
    "misa_pages_fork": (_c_int, [_p] * 3 + [_c_int] * 3 + [_p] * 4 + [_c_sz, _p]),
    "misa_pages_compact": (_c_int, [_p] * 2 + [_c_int] * 3 + [_p, _p, _c_int] + [_p] * 5
                           + [_c_sz, _p]),
    "misa_testing_score_simt": (_c_int, [_p, _p, _p, _p, _p, _p, _p, _c_int, _c_int, _c_int,
                                         _c_int, _c_i64, _c_int, _c_i64, _p, _p, _c_sz, _p]),
    "misa_testing_score_rows_wait_expiry": (_c_int, [_p, _p, _p, _p, _p, _c_int, _c_int, _c_int,
                                                     _c_int, _c_i64, _c_int, _p, _p, _c_sz,
                                                     ctypes.c_longlong, _c_int, _p]),
    "misa_testing_score_rows_timed": (_c_int, [_p, _p, _p, _p, _p, _c_int, _c_int, _c_int,
                                               _c_int, _c_i64, _c_int, _p, _p, _c_sz,
                                               ctypes.POINTER(ctypes.c_float), _p]),
    "misa_status_string": (ctypes.c_char_p, [_c_int]),
    "misa_check_device_status": (_c_int, [_p, _p]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype, _f.argtypes = _res, _args

OP_ROUTE_HEADS, OP_SCORE_TOPK, OP_DSA_TOPK, OP_DAGGER_RERANK, OP_SCORE_ROWS = 1, 2, 3, 4, 5
OP_HISA_TOPK = 6
OP_PAGES_RESIZE, OP_PAGES_FORK, OP_PAGES_COMPACT = 7, 8, 9
HEAD_DIM = 128


class MisaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: status {status} ({_lib.misa_status_string(status).decode()})")


def declared_symbols() -> list[str]:
    """Function names declared in the headers under include/ (misa.h and misa_testing.h)."""
    names = set()
    for f in sorted(os.listdir(INCLUDE_DIR)):
        if not f.endswith(".h"):
            continue
        text = open(os.path.join(INCLUDE_DIR, f)).read()
        text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
        names |= set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", text))
    return sorted(names - {"if", "sizeof", "defined"})


def library() -> ctypes.CDLL:
    return _lib


def _check(fn: str, status: int):
    if status != 0:
        raise MisaError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    # the raw handle of torch.cuda.current_stream(), without building the Python stream object
    # (0.2 against 3.4 us a call)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _bits(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"{name} must be bf16 (or its int16 bit pattern), got {t.dtype}")
    return _dev(t, name)


def _dev(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


class _Workspace:
    """One zero-initialised scratch buffer per device, grown on demand.

    Every call on a device uses this buffer, so (as the C ABI requires of one workspace)
    calls issued on different streams must not overlap on the GPU: synchronise the streams
    between them, or call the C entry points with a workspace per stream.  A buffer that a
    captured graph uses is kept for good when a larger one takes its place; make a call of a
    graph's sizes before its capture, so that the buffer is none of the graph's own memory."""

    _HEADER = 256      # bytes, with the status word

    def __init__(self):
        self._buf = {}
        self._captured = {}      # buffers that graphs hold, by device
        self._lock = threading.Lock()

    def get(self, nbytes: int, device) -> torch.Tensor:
        dev = torch.device(device)
        capturing = torch.cuda.is_current_stream_capturing()
        with self._lock:
            held = self._captured.setdefault(dev.index, [])
            b = self._buf.get(dev.index)
            if b is None or b.numel() < nbytes:
                old, b = b, torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
                if old is not None and not any(x is old for x in held):
                    if capturing:
                        held.append(old)
                    else:       # a condition recorded there moves along
                        b[:self._HEADER] = old[:self._HEADER]
                self._buf[dev.index] = b
            if capturing and not any(x is b for x in held):
                held.append(b)
            return b

    def words(self, dev: torch.device) -> list[torch.Tensor]:
        """Buffers that may hold a condition: the present one and those of captured graphs."""
        b = self.get(self._HEADER, dev)
        with self._lock:
            return [b] + [x for x in self._captured.get(dev.index, ()) if x is not b]


_WS = _Workspace()


def workspace(nbytes: int, device) -> torch.Tensor:
    return _WS.get(nbytes, device)


def misa_workspace_size(op, nseq, T, H, d, L, B, h, topk, kprime) -> int:
    return int(_lib.misa_workspace_size(op, nseq, T, H, d, L, B, h, topk, kprime))


class _Status:
    """The device status word of the paged-cache calls, one per device, kept for good: captured
    graphs hold its address.  The calls only ever write to it atomically, so streams share it."""

    def __init__(self):
        self._word = {}
        self._lock = threading.Lock()

    def get(self, device: torch.device) -> torch.Tensor:
        w = self._word.get(device.index)
        if w is None:
            with self._lock:
                w = self._word.get(device.index)
                if w is None:
                    if torch.cuda.is_current_stream_capturing():
                        raise RuntimeError("the first paged-cache call on a device allocates its "
                                           "status word: make one before capturing a graph")
                    w = torch.zeros(64, dtype=torch.int32, device=device)
                    torch.cuda.current_stream(device).synchronize()   # zero for every stream
                    self._word[device.index] = w
        return w

    def find(self, index: int) -> torch.Tensor | None:
        return self._word.get(index)


_STATUS = _Status()


def misa_check_device_status(device=None) -> int:
    """Synchronise the current stream, read and clear the status words (the workspace's, then the
    paged-cache calls'); raise if one is set.  Where several are, the others stay for the next call."""
    dev = torch.device(device if device is not None else "cuda")
    if dev.index is None:      # the current device, whose buffers are kept under its number
        dev = torch.device("cuda", torch.cuda.current_device())
    for word in (*_WS.words(dev), _STATUS.find(dev.index)):
        if word is not None:
            _check("misa_check_device_status",
                   int(_lib.misa_check_device_status(_ptr(word), _stream())))
    return 0


def misa_pool_keys(k: torch.Tensor, B: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Mean-pool k [nseq, L, d] (bf16) into fp32 [nseq, ceil(L/B), d] (Eq. 4)."""
    k = _bits(k, "k")
    nseq, L, d = k.shape
    M = -(-L // B)
    if out is None:
        out = torch.empty((nseq, M, d), dtype=torch.float32, device=k.device)
    _check("misa_pool_keys",
           _lib.misa_pool_keys(_ptr(k), nseq, L, d, B, _ptr(out), _stream()))
    return out


def misa_pool_keys_range(k: torch.Tensor, B: int, k_pool: torch.Tensor, s_begin: int,
                         s_end: int) -> torch.Tensor:
    """Recompute, in place, the pooled blocks of k_pool that meet tokens [s_begin, s_end)
    of every sequence (the keys there changed); other blocks are left as they are."""
    k = _bits(k, "k")
    nseq, L, d = k.shape
    k_pool = _dev(k_pool, "k_pool", torch.float32)
    if tuple(k_pool.shape) != (nseq, -(-L // B), d):
        raise ValueError(f"k_pool must be [{nseq}, {-(-L // B)}, {d}], got {tuple(k_pool.shape)}")
    _check("misa_pool_keys_range",
           _lib.misa_pool_keys_range(_ptr(k), nseq, L, d, B, int(s_begin), int(s_end),
                                     _ptr(k_pool), _stream()))
    return k_pool


def misa_route_heads(q, w, k, k_pool, pos, B: int, h: int, return_E: bool = False,
                     heads: torch.Tensor | None = None, E: torch.Tensor | None = None):
    """Route each query to its top-h heads by block-pooled energy (Eqs. 7-8)."""
    q, k = _bits(q, "q"), _bits(k, "k")
    w = _dev(w, "w", torch.float32)
    k_pool = _dev(k_pool, "k_pool", torch.float32)
    pos = _dev(pos, "pos", torch.int32)
    nseq, T, H, d = q.shape
    L = k.shape[1]
    if heads is None:
        heads = torch.empty((nseq, T, h), dtype=torch.int32, device=q.device)
    if return_E and E is None:
        E = torch.empty((nseq, T, H), dtype=torch.float32, device=q.device)
    nb = misa_workspace_size(OP_ROUTE_HEADS, nseq, T, H, d, L, B, h, 1, 1)
    if nb == 0:
        raise MisaError("misa_workspace_size", 1)
    ws = _WS.get(nb, q.device)
    _check("misa_route_heads",
           _lib.misa_route_heads(_ptr(q), _ptr(w), _ptr(k), _ptr(k_pool), _ptr(pos), nseq, T, H,
                                 d, L, B, h, _ptr(heads), _ptr(E), _ptr(ws), ws.numel(),
                                 _stream()))
    return (heads, E) if return_E else heads


def _outs(rows_shape, topk, device, idx, vals, want_vals):
    if idx is None:
        idx = torch.empty(rows_shape + (topk,), dtype=torch.int32, device=device)
    if want_vals and vals is None:
        vals = torch.empty(rows_shape + (topk,), dtype=torch.float32, device=device)
    return idx, vals


def misa_score_topk(q, w, k, heads, pos, topk: int, return_vals: bool = True,
                    scores: torch.Tensor | None = None, idx=None, vals=None):
    """Routed scores over each query's prefix and their top-k (Eqs. 9-10)."""
    q, k = _bits(q, "q"), _bits(k, "k")
    w = _dev(w, "w", torch.float32)
    heads = _dev(heads, "heads", torch.int32)
    pos = _dev(pos, "pos", torch.int32)
    nseq, T, H, d = q.shape
    L = k.shape[1]
    h = heads.shape[-1]
    idx, vals = _outs((nseq, T), topk, q.device, idx, vals, return_vals)
    if scores is not None:
        _dev(scores, "scores", torch.float32)
    nb = misa_workspace_size(OP_SCORE_TOPK, nseq, T, H, d, L, 1, h, topk, topk)
    if nb == 0:
        raise MisaError("misa_workspace_size", 1)
    ws = _WS.get(nb, q.device)
    _check("misa_score_topk",
           _lib.misa_score_topk(_ptr(q), _ptr(w), _ptr(k), _ptr(heads), _ptr(pos), nseq, T, H, d,
                                L, h, topk, _ptr(idx), _ptr(vals), _ptr(scores), _ptr(ws),
                                ws.numel(), _stream()))
    return (idx, vals) if return_vals else idx


def dsa_score_topk(q, w, k, pos, topk: int, return_vals: bool = True,
                   scores: torch.Tensor | None = None, idx=None, vals=None):
    """Dense DSA indexer scores (all heads, Eq. 1) and their top-k (Eq. 2)."""
    q, k = _bits(q, "q"), _bits(k, "k")
    w = _dev(w, "w", torch.float32)
    pos = _dev(pos, "pos", torch.int32)
    nseq, T, H, d = q.shape
    L = k.shape[1]
    idx, vals = _outs((nseq, T), topk, q.device, idx, vals, return_vals)
    if scores is not None:
        _dev(scores, "scores", torch.float32)
    nb = misa_workspace_size(OP_DSA_TOPK, nseq, T, H, d, L, 1, 1, topk, topk)
    if nb == 0:
        raise MisaError("misa_workspace_size", 1)
    ws = _WS.get(nb, q.device)
    _check("dsa_score_topk",
           _lib.dsa_score_topk(_ptr(q), _ptr(w), _ptr(k), _ptr(pos), nseq, T, H, d, L, topk,
                               _ptr(idx), _ptr(vals), _ptr(scores), _ptr(ws), ws.numel(),
                               _stream()))
    return (idx, vals) if return_vals else idx


def misa_score_rows(q, w, k, heads, pos, scores: torch.Tensor | None = None):
    """Token scores without selection: routed (Eq. 9) when heads is given, dense (Eq. 1)
    when heads is None.  Returns fp32 [nseq, T, L]; entries past each query's position
    are left as they were."""
    q, k = _bits(q, "q"), _bits(k, "k")
    w = _dev(w, "w", torch.float32)
    pos = _dev(pos, "pos", torch.int32)
    nseq, T, H, d = q.shape
    L = k.shape[1]
    if heads is not None:
        heads = _dev(heads, "heads", torch.int32)
    h = heads.shape[-1] if heads is not None else H
    if scores is None:
        scores = torch.empty((nseq, T, L), dtype=torch.float32, device=q.device)
    _dev(scores, "scores", torch.float32)
    nb = misa_workspace_size(OP_SCORE_ROWS, nseq, T, H, d, L, 1, h, 1, 1)
    if nb == 0:
        raise MisaError("misa_workspace_size", 1)
    ws = _WS.get(nb, q.device)
    _check("misa_score_rows",
           _lib.misa_score_rows(_ptr(q), _ptr(w), _ptr(k), _ptr(heads), _ptr(pos), nseq, T, H, d,
                                L, h, _ptr(scores), _ptr(ws), ws.numel(), _stream()))
    return scores


def misa_dagger_rerank(q, w, k, pos, cand, topk: int, return_vals: bool = True, idx=None,
                       vals=None):
    """Re-score candidates with all heads and keep the top-k (Eq. 12)."""
    q, k = _bits(q, "q"), _bits(k, "k")
    w = _dev(w, "w", torch.float32)
    pos = _dev(pos, "pos", torch.int32)
    cand = _dev(cand, "cand", torch.int32)
    nseq, T, H, d = q.shape
    L = k.shape[1]
    kprime = cand.shape[-1]
    idx, vals = _outs((nseq, T), topk, q.device, idx, vals, return_vals)
    nb = misa_workspace_size(OP_DAGGER_RERANK, nseq, T, H, d, L, 1, 1, topk, kprime)
    if nb == 0:
        raise MisaError("misa_workspace_size", 1)
    ws = _WS.get(nb, q.device)
    _check("misa_dagger_rerank",
           _lib.misa_dagger_rerank(_ptr(q), _ptr(w), _ptr(k), _ptr(pos), _ptr(cand), nseq, T, H,
                                   d, L, kprime, topk, _ptr(idx), _ptr(vals), _ptr(ws),
                                   ws.numel(), _stream()))
    return (idx, vals) if return_vals else idx


def hisa_block_filter_topk(q, w, k, k_pool, pos, B: int, m: int, topk: int,
                           return_vals: bool = True, return_blocks: bool = False, idx=None,
                           vals=None, blocks=None):
    """HISA-style token-axis filter: keep each query's m blocks with the largest
    head-summed affinity G[b] = sum_j w_j ReLU(q_j . kp_b), then the top-k of the
    all-head score (Eq. 1) over their tokens.  k_pool: misa_pool_keys(k, B)."""
    q, k = _bits(q, "q"), _bits(k, "k")
    w = _dev(w, "w", torch.float32)
    k_pool = _dev(k_pool, "k_pool", torch.float32)
    pos = _dev(pos, "pos", torch.int32)
    nseq, T, H, d = q.shape
    L = k.shape[1]
    idx, vals = _outs((nseq, T), topk, q.device, idx, vals, return_vals)
    if return_blocks and blocks is None:
        blocks = torch.empty((nseq, T, m), dtype=torch.int32, device=q.device)
    nb = misa_workspace_size(OP_HISA_TOPK, nseq, T, H, d, L, B, m, topk, 0)
    if nb == 0:
        raise MisaError("misa_workspace_size", 1)
    ws = _WS.get(nb, q.device)
    _check("hisa_block_filter_topk",
           _lib.hisa_block_filter_topk(_ptr(q), _ptr(w), _ptr(k), _ptr(k_pool), _ptr(pos), nseq,
                                       T, H, d, L, B, m, topk, _ptr(idx), _ptr(vals),
                                       _ptr(blocks), _ptr(ws), ws.numel(), _stream()))
    out = (idx, vals) if return_vals else (idx,)
    if return_blocks:
        out = out + (blocks,)
    return out if len(out) > 1 else out[0]


def misa_score_topk_noalloc(q, w, k, heads, pos, topk: int, return_vals: bool = True, idx=None,
                            vals=None, device_status=None):
    """misa_score_topk for callers that cannot allocate: the library uses its own fixed
    16 MiB scratch (nseq * T * L <= 4,194,304) instead of a workspace.  Outputs are
    allocated here only when not passed in; pass idx / vals / device_status to make
    the call allocation-free from Python too.  Calls whose GPU work overlaps race on
    the shared scratch and must be serialised."""
    q, k = _bits(q, "q"), _bits(k, "k")
    w = _dev(w, "w", torch.float32)
    heads = _dev(heads, "heads", torch.int32)
    pos = _dev(pos, "pos", torch.int32)
    nseq, T, H, d = q.shape
    L = k.shape[1]
    h = heads.shape[-1]
    idx, vals = _outs((nseq, T), topk, q.device, idx, vals, return_vals)
    _check("misa_score_topk_noalloc",
           _lib.misa_score_topk_noalloc(_ptr(q), _ptr(w), _ptr(k), _ptr(heads), _ptr(pos), nseq,
                                        T, H, d, L, h, topk, _ptr(idx), _ptr(vals),
                                        _ptr(device_status), _stream()))
    return (idx, vals) if return_vals else idx


# ----------------------------------------------------------------- paged key-value cache
# Scratch is a fresh tensor of torch's caching allocator per call: it belongs to the call's
# stream, and under graph capture to the graph, so neither streams nor graphs share it.

_CACHE_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


@functools.lru_cache(maxsize=1024)
def _attention_ws(*sizes) -> int:
    return int(_lib.misa_paged_attention_workspace_size(*sizes))


@functools.lru_cache(maxsize=1024)
def _pages_ws(*sizes) -> int:
    return int(_lib.misa_pages_workspace_size(*sizes))


def _scratch(nbytes: int, like: torch.Tensor):
    """nbytes (a multiple of 256) beside the int32 tensor `like`, or None for 0."""
    return like.new_empty(nbytes // 4) if nbytes else None


def _shape(t: torch.Tensor, shape: tuple, name: str):
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _cache(k_cache, v_cache, page_table, pos):
    """Checks what attention and append share; returns the dtype code and the cache's sizes."""
    if k_cache.dtype not in _CACHE_DTYPES:
        raise TypeError(f"k_cache must be bf16 or fp16, got {k_cache.dtype}")
    _dev(k_cache, "k_cache")
    _dev(v_cache, "v_cache", k_cache.dtype)
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, page_size, Hkv, d]")
    _shape(v_cache, tuple(k_cache.shape), "v_cache")
    _dev(page_table, "page_table", torch.int32)
    _dev(pos, "pos", torch.int32)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [nseq, max_pages]")
    return _CACHE_DTYPES[k_cache.dtype], k_cache.shape


def misa_paged_attention(q, k_cache, v_cache, page_table, pos, idx=None,
                         scale: float | None = None, return_lse: bool = False, out=None,
                         lse=None):
    """Attention of new tokens over a paged cache: each query's prefix 0 .. pos, or the tokens
    of its idx row (an indexer's selection, -1 padded).

    q [nseq, T, Hq, d], k_cache / v_cache [num_pages, page_size, Hkv, d] (bf16 or fp16, one type),
    page_table int32 [nseq, max_pages], pos int32 [nseq, T] (-1: a padded row), idx int32
    [nseq, T, topk]; scale defaults to d ** -0.5.  Returns out [nseq, T, Hq, d], and with
    return_lse also lse fp32 [nseq, T, Hq]."""
    code, (num_pages, page_size, Hkv, d) = _cache(k_cache, v_cache, page_table, pos)
    _dev(q, "q", k_cache.dtype)
    if q.dim() != 4:
        raise ValueError("q must be [nseq, T, Hq, d]")
    nseq, T, Hq, _ = q.shape
    _shape(q, (nseq, T, Hq, d), "q")
    _shape(pos, (nseq, T), "pos")
    if page_table.shape[0] != nseq:
        raise ValueError(f"page_table must have {nseq} rows, got {page_table.shape[0]}")
    topk = 0
    if idx is not None:
        _dev(idx, "idx", torch.int32)
        topk = idx.shape[-1]
        _shape(idx, (nseq, T, topk), "idx")
        if topk == 0:
            raise ValueError("idx must list at least one token")
    if out is None:
        out = torch.empty_like(q)
    else:
        _dev(out, "out", q.dtype)
        _shape(out, tuple(q.shape), "out")
    if lse is not None:
        _dev(lse, "lse", torch.float32)
        _shape(lse, (nseq, T, Hq), "lse")
    elif return_lse:
        lse = torch.empty((nseq, T, Hq), dtype=torch.float32, device=q.device)
    max_pages = page_table.shape[1]
    nb = _attention_ws(nseq, T, Hq, Hkv, d, page_size, max_pages, topk)
    ws = _scratch(nb, pos)
    _check("misa_paged_attention",
           _lib.misa_paged_attention(
               q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
               pos.data_ptr(), _ptr(idx), code, nseq, T, Hq, Hkv, d, num_pages, page_size,
               max_pages, topk, d ** -0.5 if scale is None else scale, out.data_ptr(),
               _ptr(lse), _STATUS.get(q.device).data_ptr(), _ptr(ws), nb, _stream()))
    return (out, lse) if return_lse else out


def misa_paged_append(k_new, v_new, pos, page_table, k_cache, v_cache):
    """Write the keys and values of new tokens ([nseq, T, Hkv, d]) into their pages: row (n, t)
    becomes token pos[n, t] of sequence n (-1: skipped).  In place; returns the caches."""
    code, (num_pages, page_size, Hkv, d) = _cache(k_cache, v_cache, page_table, pos)
    _dev(k_new, "k_new", k_cache.dtype)
    _dev(v_new, "v_new", k_cache.dtype)
    nseq, T = pos.shape
    _shape(k_new, (nseq, T, Hkv, d), "k_new")
    _shape(v_new, (nseq, T, Hkv, d), "v_new")
    if page_table.shape[0] != nseq:
        raise ValueError(f"page_table must have {nseq} rows, got {page_table.shape[0]}")
    _check("misa_paged_append",
           _lib.misa_paged_append(
               k_new.data_ptr(), v_new.data_ptr(), pos.data_ptr(), page_table.data_ptr(), code,
               nseq, T, Hkv, d, num_pages, page_size, page_table.shape[1], k_cache.data_ptr(),
               v_cache.data_ptr(), _STATUS.get(k_cache.device).data_ptr(), _stream()))
    return k_cache, v_cache


def _upkeep(op, page_table, refs, out_table, out_refs):
    """Checks of the table and the counts; returns the outputs, scratch and its size."""
    _dev(page_table, "page_table", torch.int32)
    _dev(refs, "refs", torch.int32)
    if page_table.dim() != 2 or refs.dim() != 1:
        raise ValueError("page_table must be [nseq, max_pages] and refs [num_pages]")
    if out_table is None:
        out_table = torch.empty_like(page_table)
    else:
        _dev(out_table, "out_table", torch.int32)
        _shape(out_table, tuple(page_table.shape), "out_table")
    if out_refs is None:
        out_refs = torch.empty_like(refs)
    else:
        _dev(out_refs, "out_refs", torch.int32)
        _shape(out_refs, tuple(refs.shape), "out_refs")
    nseq, max_pages = page_table.shape
    nb = _pages_ws(op, nseq, max_pages, refs.shape[0])
    return out_table, out_refs, _scratch(nb, refs), nb


def _pools(pools, num_pages: int):
    n = len(pools)
    if n == 0:
        return None, None, 0
    for i, t in enumerate(pools):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"pools[{i}] must be a contiguous CUDA tensor")
        if t.dim() == 0 or t.shape[0] != num_pages:
            raise ValueError(f"pools[{i}] must have {num_pages} pages")
    return (array.array("Q", [t.data_ptr() for t in pools]),
            array.array("q", [t.nbytes // num_pages for t in pools]), n)


def _address(a: array.array | None) -> int | None:
    return None if a is None else a.buffer_info()[0]


def misa_pages_resize(page_table, refs, old_len, new_len, page_size: int, pools=(),
                      out_table=None, out_refs=None):
    """Give every sequence the pages for new_len tokens where it held those for old_len: take
    free pages (lowest first), copy a shared, partly filled last page in every pool before it is
    written, let go of pages.  Returns (page_table, refs); pass out_table=page_table,
    out_refs=refs for in place.  With too few free pages nothing changes, and
    misa_check_device_status reports it."""
    out_table, out_refs, ws, nb = _upkeep(OP_PAGES_RESIZE, page_table, refs, out_table,
                                          out_refs)
    nseq, max_pages = page_table.shape
    for t, name in ((old_len, "old_len"), (new_len, "new_len")):
        _dev(t, name, torch.int32)
        _shape(t, (nseq,), name)
    ptrs, sizes, n = _pools(pools, refs.shape[0])
    _check("misa_pages_resize",
           _lib.misa_pages_resize(
               page_table.data_ptr(), refs.data_ptr(), old_len.data_ptr(), new_len.data_ptr(),
               nseq, max_pages, refs.shape[0], page_size, _address(ptrs), _address(sizes), n,
               out_table.data_ptr(), out_refs.data_ptr(), _STATUS.get(refs.device).data_ptr(),
               _ptr(ws), nb, _stream()))
    return out_table, out_refs


def misa_pages_fork(page_table, refs, parent, out_table=None, out_refs=None):
    """Row n takes the pages of row parent[n] (-1: none), all rows at once; refs follow and no
    page is copied.  Returns (page_table, refs)."""
    out_table, out_refs, ws, nb = _upkeep(OP_PAGES_FORK, page_table, refs, out_table, out_refs)
    nseq, max_pages = page_table.shape
    _dev(parent, "parent", torch.int32)
    _shape(parent, (nseq,), "parent")
    _check("misa_pages_fork",
           _lib.misa_pages_fork(
               page_table.data_ptr(), refs.data_ptr(), parent.data_ptr(), nseq, max_pages,
               refs.shape[0], out_table.data_ptr(), out_refs.data_ptr(),
               _STATUS.get(refs.device).data_ptr(), _ptr(ws), nb, _stream()))
    return out_table, out_refs


def misa_pages_compact(page_table, refs, pools=(), out_table=None, out_refs=None, n_live=None):
    """Move the pages in use to the front of the pools (contents, table and counts).  Returns
    (page_table, refs, n_live): n_live int32 [1], the pages in use."""
    out_table, out_refs, ws, nb = _upkeep(OP_PAGES_COMPACT, page_table, refs, out_table,
                                          out_refs)
    nseq, max_pages = page_table.shape
    if n_live is None:
        n_live = refs.new_empty(1)
    else:
        _dev(n_live, "n_live", torch.int32)
        _shape(n_live, (1,), "n_live")
    ptrs, sizes, n = _pools(pools, refs.shape[0])
    _check("misa_pages_compact",
           _lib.misa_pages_compact(
               page_table.data_ptr(), refs.data_ptr(), nseq, max_pages, refs.shape[0],
               _address(ptrs), _address(sizes), n, out_table.data_ptr(), out_refs.data_ptr(), n_live.data_ptr(),
               _STATUS.get(refs.device).data_ptr(), _ptr(ws), nb, _stream()))
    return out_table, out_refs, n_live


# ----------------------------------------------------------------- test-only entry points
# (include/misa_testing.h): the CUDA-core scorer on its own, and the tensor-core scorer
# with shortened wait bounds and one key tile never loaded.

def misa_testing_score_simt(q, w, k, heads, pos, gather_ids=None, gather_len=None,
                            scores: torch.Tensor | None = None):
    """The CUDA-core scorer: Eq. (9) under heads (Eq. 1 with heads None) over each
    query's prefix, or over gather_ids[row, :gather_len[row]] when given.  Returns fp32
    [nseq, T, L] (prefix) or [nseq, T, kprime] (gather)."""
    q, k = _bits(q, "q"), _bits(k, "k")
    w = _dev(w, "w", torch.float32)
    pos = _dev(pos, "pos", torch.int32)
    nseq, T, H, d = q.shape
    L = k.shape[1]
    if heads is not None:
        heads = _dev(heads, "heads", torch.int32)
    h = heads.shape[-1] if heads is not None else H
    if gather_ids is not None:
        gather_ids = _dev(gather_ids, "gather_ids", torch.int32)
        gather_len = _dev(gather_len, "gather_len", torch.int32)
        stride = gather_ids.shape[-1]
    else:
        stride = L
    if scores is None:
        scores = torch.full((nseq, T, stride), float("nan"), dtype=torch.float32,
                            device=q.device)
    ws = _WS.get(256, q.device)
    _check("misa_testing_score_simt",
           _lib.misa_testing_score_simt(_ptr(q), _ptr(w), _ptr(k), _ptr(heads), _ptr(pos),
                                        _ptr(gather_ids), _ptr(gather_len), nseq, T, H, d, L, h,
                                        stride, _ptr(scores), _ptr(ws), ws.numel(), _stream()))
    return scores


def misa_testing_score_rows_wait_expiry(q, w, k, heads, pos, wait_cycles: int, skip_tile: int,
                                        scores: torch.Tensor | None = None):
    """misa_score_rows with every wait bounded by wait_cycles and key tile skip_tile never
    loaded (-1: none).  Read the outcome with misa_check_device_status."""
    q, k = _bits(q, "q"), _bits(k, "k")
    w = _dev(w, "w", torch.float32)
    pos = _dev(pos, "pos", torch.int32)
    nseq, T, H, d = q.shape
    L = k.shape[1]
    if heads is not None:
        heads = _dev(heads, "heads", torch.int32)
    h = heads.shape[-1] if heads is not None else H
    if scores is None:
        scores = torch.full((nseq, T, L), float("nan"), dtype=torch.float32, device=q.device)
    nb = misa_workspace_size(OP_SCORE_ROWS, nseq, T, H, d, L, 1, h, 1, 1)
    if nb == 0:
        raise MisaError("misa_workspace_size", 1)
    ws = _WS.get(nb, q.device)
    _check("misa_testing_score_rows_wait_expiry",
           _lib.misa_testing_score_rows_wait_expiry(_ptr(q), _ptr(w), _ptr(k), _ptr(heads),
                                                    _ptr(pos), nseq, T, H, d, L, h,
                                                    _ptr(scores), _ptr(ws), ws.numel(),
                                                    int(wait_cycles), int(skip_tile), _stream()))
    return scores


def misa_testing_score_rows_timed(q, w, k, heads, pos, scores: torch.Tensor | None = None):
    """misa_score_rows on the tensor-core scorer; returns the device milliseconds of its
    scoring kernel alone (CUDA events around that launch; the call waits for it)."""
    q, k = _bits(q, "q"), _bits(k, "k")
    w = _dev(w, "w", torch.float32)
    pos = _dev(pos, "pos", torch.int32)
    nseq, T, H, d = q.shape
    L = k.shape[1]
    if heads is not None:
        heads = _dev(heads, "heads", torch.int32)
    h = heads.shape[-1] if heads is not None else H
    if scores is None:
        scores = torch.empty((nseq, T, L), dtype=torch.float32, device=q.device)
    nb = misa_workspace_size(OP_SCORE_ROWS, nseq, T, H, d, L, 1, h, 1, 1)
    if nb == 0:
        raise MisaError("misa_workspace_size", 1)
    ws = _WS.get(nb, q.device)
    ms = ctypes.c_float(0.0)
    _check("misa_testing_score_rows_timed",
           _lib.misa_testing_score_rows_timed(_ptr(q), _ptr(w), _ptr(k), _ptr(heads), _ptr(pos),
                                              nseq, T, H, d, L, h, _ptr(scores), _ptr(ws),
                                              ws.numel(), ctypes.byref(ms), _stream()))
    return float(ms.value)


def misa_testing_paged_attention_wait_expiry(q, k_cache, v_cache, page_table, pos,
                                             wait_cycles: int, skip_tile: int):
    """misa_paged_attention over prefixes, in its form for many query rows, with every wait
    bounded by wait_cycles and the keys of the first CTA's tile skip_tile never loaded (-1:
    none).  Read the outcome with misa_check_device_status."""
    code, (num_pages, page_size, Hkv, d) = _cache(k_cache, v_cache, page_table, pos)
    _dev(q, "q", k_cache.dtype)
    nseq, T, Hq, _ = q.shape
    out = torch.zeros_like(q)
    max_pages = page_table.shape[1]
    nb = _attention_ws(nseq, T, Hq, Hkv, d, page_size, max_pages, 0)
    ws = torch.zeros(max(nb, 4) // 4, dtype=torch.int32, device=q.device)
    _check("misa_testing_paged_attention_wait_expiry",
           _lib.misa_testing_paged_attention_wait_expiry(
               q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
               pos.data_ptr(), None, code, nseq, T, Hq, Hkv, d, num_pages, page_size, max_pages,
               0, d ** -0.5, out.data_ptr(), None, _STATUS.get(q.device).data_ptr(), _ptr(ws), nb,
               int(wait_cycles), int(skip_tile), _stream()))
    return out
