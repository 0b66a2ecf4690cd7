"""ctypes binding of libecho -- argument marshalling only.

Every call takes torch CUDA tensors (or None where the C ABI allows NULL),
passes their device addresses and the current CUDA stream to the library and
returns.  Nothing here computes: all work runs in the library's kernels.  The
library must be built (``build()``); there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

ECHO_OK, ECHO_EINVAL, ECHO_ECAPACITY, ECHO_EUNSUPPORTED, ECHO_ECUDA, ECHO_ETOOLARGE = 0, -1, -2, -3, -4, -5
PREFILL_STATIC_SCRATCH_BYTES = 32 << 20
ST_TIMEOUT, ST_NAN, ST_NOSLOT, ST_BADDATA, ST_FULL = 0x1, 0x2, 0x4, 0x8, 0x10
STAT_TOPK_FALLBACK, STAT_BOUNDARY_MAX, STAT_EARLY, STAT_MISSES, STAT_EARLY_USED, STAT_CAND_MISS = 0, 1, 2, 3, 4, 5
STAT_REVIVED = 6
STATS_N = 8
HEADS, DIM, MAX_REQUESTS = 64, 128, 4096
CACHE_HOLD_EARLY, CACHE_LAZY = 1, 2   # echo_cache_step flags
TOPK_CACHED_MAX_SLOTS = 32768  # C limit of echo_topk_select_cached and of the cached form of echo_topk_select_cands
CAND_CAP = 16384             # candidate-list entries per request top-k keeps in shared memory
TREE_MAX_WORDS, TREE_MAX_NODES = 32, 1024   # words of a tree's masks, its nodes
DTYPE_F32, DTYPE_BF16, MAX_VOCAB = 0, 1, 1 << 24   # echo_draft_verify
POOL_MAX_PAGES = 1 << 24
EARLY_FETCH_BLOCKS = 24      # CTAs of the early-fetch and late-recall kernels

EXPORTS = ("echo_above_words", "echo_append_tokens", "echo_cache_release", "echo_cache_step", "echo_cache_step_resolved",
           "echo_debug_stall_epilogue", "echo_debug_wait_limit", "echo_device_sm_count", "echo_draft_verify",
           "echo_early_fetch", "echo_evict_select", "echo_evict_select_resident", "echo_host_device_alias", "echo_index_scores", "echo_index_scores_cands", "echo_mla_chunk",
           "echo_mla_chunk_workspace_size", "echo_mla_decode", "echo_mla_mass",
           "echo_mla_mass_workspace_size", "echo_mla_tree", "echo_pages_compact", "echo_pages_fork", "echo_pages_free",
           "echo_pages_reserve", "echo_pages_workspace_size", "echo_pool_above", "echo_pool_select", "echo_rows_keep",
           "echo_pool_slots", "echo_prefill_block",
           "echo_prefill_block_static", "echo_prefill_scores", "echo_prefill_workspace_size", "echo_quantize_q", "echo_seed_early",
           "echo_topk_select", "echo_topk_select_cached", "echo_topk_select_cands",
           "echo_tree_masks")

_vp = ctypes.c_void_p


class EchoCacheStruct(ctypes.Structure):
    _fields_ = [("tok2slot", _vp), ("slot2tok", _vp), ("freebits", _vp), ("miss_tok", _vp),
                ("miss_slot", _vp), ("miss_cnt", _vp), ("early_tok", _vp), ("early_slot", _vp),
                ("early_cnt", _vp), ("free_snap", _vp), ("host_kv", _vp), ("dev_kv", _vp), ("row_bytes", ctypes.c_int64),
                ("C", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class EchoCandsStruct(ctypes.Structure):
    _fields_ = [("key", _vp), ("idx", _vp), ("cnt", _vp), ("cut", _vp), ("cap", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class EchoPagesStruct(ctypes.Structure):
    _fields_ = [("page_tab", _vp), ("kv", _vp), ("kv_rows", ctypes.c_int64), ("req_rows", ctypes.c_int64),
                ("page", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class EchoPagePoolStruct(ctypes.Structure):
    _fields_ = [("page_tab", _vp), ("refs", _vp), ("kv", _vp), ("n_pages", ctypes.c_int64), ("row_bytes", ctypes.c_int64),
                ("layer_bytes", ctypes.c_int64), ("layers", ctypes.c_int32), ("page", ctypes.c_int32)]


class EchoError(RuntimeError):
    def __init__(self, call, rc):
        super().__init__(f"{call} returned {rc}")
        self.rc = rc


_lock = threading.Lock()
_lib = None


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libecho.so (raises when it is missing and not built)."""
    global _lib
    if _lib is not None:  # (set once, when it is complete)
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_build.LIB):
            if not build_if_missing:
                raise RuntimeError(f"libecho is not built ({_build.LIB}); run "
                                   "python -m sparse_attention_kv_echo_gb300.build")
            _build.build()
        L = ctypes.CDLL(_build.LIB)
        i32, i64, f32 = ctypes.c_int, ctypes.c_int64, ctypes.c_float
        L.echo_quantize_q.restype = i32
        L.echo_quantize_q.argtypes = [i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
        L.echo_above_words.restype = ctypes.c_size_t
        L.echo_above_words.argtypes = [i32, i64]
        L.echo_index_scores.restype = i32
        L.echo_index_scores.argtypes = [i32, _vp, _vp, i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                        ctypes.POINTER(EchoCacheStruct), i32, _vp, _vp]
        L.echo_index_scores_cands.restype = i32
        L.echo_index_scores_cands.argtypes = [i32, _vp, _vp, i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                              ctypes.POINTER(EchoCacheStruct), ctypes.POINTER(EchoCandsStruct),
                                              i32, _vp, _vp]
        L.echo_topk_select_cands.restype = i32
        L.echo_topk_select_cands.argtypes = [i32, _vp, _vp, i64, _vp, i32, _vp, _vp, f32,
                                             ctypes.POINTER(EchoCandsStruct), _vp, _vp, _vp, i32,
                                             ctypes.POINTER(EchoCacheStruct), _vp, _vp, _vp, _vp]
        L.echo_early_fetch.restype = i32
        L.echo_early_fetch.argtypes = [i32, _vp, _vp, i64, _vp, i32, ctypes.POINTER(EchoCacheStruct), _vp, _vp]
        L.echo_topk_select.restype = i32
        L.echo_topk_select.argtypes = [i32, _vp, _vp, i64, _vp, i32, _vp, _vp, f32, _vp, _vp, _vp, _vp, _vp]
        L.echo_cache_step.restype = i32
        L.echo_cache_step.argtypes = [i32, _vp, _vp, i64, _vp, i32, _vp, i32, ctypes.POINTER(EchoCacheStruct), _vp,
                                      _vp, _vp, _vp, _vp, i32]
        L.echo_mla_decode.restype = i32
        L.echo_mla_decode.argtypes = [i32, i32, _vp, _vp, _vp, i64, f32, _vp, _vp, _vp, _vp]
        pages = ctypes.POINTER(EchoPagesStruct)
        L.echo_mla_chunk_workspace_size.restype = ctypes.c_size_t
        L.echo_mla_chunk_workspace_size.argtypes = [i64, i32, i32]
        L.echo_mla_chunk.restype = i32
        L.echo_mla_chunk.argtypes = [i32, _vp, i64, i32, _vp, _vp, _vp, i64, pages, _vp, i32, i64, i64, f32, _vp, _vp,
                                     _vp, ctypes.c_size_t, _vp, _vp]
        L.echo_mla_mass.restype = i32
        L.echo_mla_mass.argtypes = [i32, _vp, i64, i32, _vp, _vp, _vp, _vp, i64, pages, i64, i64, f32, _vp, _vp, f32,
                                    _vp, ctypes.c_size_t, _vp, _vp]
        L.echo_mla_mass_workspace_size.restype = ctypes.c_size_t
        L.echo_mla_mass_workspace_size.argtypes = [i64, i32]
        L.echo_tree_masks.restype = i32
        L.echo_tree_masks.argtypes = [i32, _vp, i64, _vp, i32, _vp, _vp, _vp, _vp]
        L.echo_mla_tree.restype = i32
        L.echo_mla_tree.argtypes = [i32, _vp, i64, i32, _vp, _vp, i32, _vp, _vp, i64, pages, f32, _vp, _vp, _vp,
                                    ctypes.c_size_t, _vp, _vp]
        L.echo_draft_verify.restype = i32
        L.echo_draft_verify.argtypes = [i32, _vp, i64, _vp, _vp, i64, i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
        pool = ctypes.POINTER(EchoPagePoolStruct)
        L.echo_pages_workspace_size.restype = ctypes.c_size_t
        L.echo_pages_workspace_size.argtypes = [i32, i64]
        L.echo_pages_reserve.restype = i32
        L.echo_pages_reserve.argtypes = [i32, _vp, _vp, _vp, i64, pool, _vp, _vp, ctypes.c_size_t, _vp, _vp]
        L.echo_pages_free.restype = i32
        L.echo_pages_free.argtypes = [i32, _vp, _vp, i64, pool, _vp, _vp]
        L.echo_pages_fork.restype = i32
        L.echo_pages_fork.argtypes = [i32, _vp, _vp, i32, _vp, _vp, i64, pool, _vp, ctypes.c_size_t, _vp, _vp]
        L.echo_pages_compact.restype = i32
        L.echo_pages_compact.argtypes = [i64, pool, _vp, _vp, ctypes.c_size_t, _vp, _vp]
        L.echo_rows_keep.restype = i32
        L.echo_rows_keep.argtypes = [i32, _vp, i64, _vp, _vp, _vp, _vp, i64, pool, _vp, _vp, _vp]
        L.echo_evict_select.restype = i32
        L.echo_evict_select.argtypes = [i32, _vp, _vp, i64, _vp, i32, _vp, i64, i64, i64, _vp, _vp, _vp, _vp, _vp]
        L.echo_evict_select_resident.restype = i32
        L.echo_evict_select_resident.argtypes = [i32, _vp, _vp, i64, _vp, _vp, i32, _vp, i64, i64, i64, _vp, _vp, _vp, _vp,
                                                 _vp]
        L.echo_cache_release.restype = i32
        L.echo_cache_release.argtypes = [i32, _vp, _vp, i64, _vp, i32, ctypes.POINTER(EchoCacheStruct), _vp, _vp, _vp]
        L.echo_pool_above.restype = i32
        L.echo_pool_above.argtypes = [i32, _vp, _vp, i64, _vp, ctypes.POINTER(EchoCacheStruct), _vp, _vp, _vp]
        L.echo_pool_select.restype = i32
        L.echo_pool_select.argtypes = [i32, _vp, _vp, i32, _vp, _vp]
        L.echo_pool_slots.restype = i32
        L.echo_pool_slots.argtypes = [i32, _vp, i32, _vp, _vp, _vp]
        L.echo_seed_early.restype = i32
        L.echo_seed_early.argtypes = [i32, _vp, _vp, i64, _vp, i32, _vp, ctypes.POINTER(EchoCacheStruct), _vp, _vp]
        L.echo_append_tokens.restype = i32
        L.echo_append_tokens.argtypes = [i32, _vp, _vp, i64, _vp, _vp, _vp, _vp, ctypes.POINTER(EchoCacheStruct),
                                         _vp, _vp]
        L.echo_topk_select_cached.restype = i32
        L.echo_topk_select_cached.argtypes = [i32, _vp, _vp, i64, _vp, i32, _vp, _vp, f32, _vp, _vp, _vp, i32,
                                              ctypes.POINTER(EchoCacheStruct), _vp, _vp, _vp, _vp]
        L.echo_cache_step_resolved.restype = i32
        L.echo_cache_step_resolved.argtypes = [i32, _vp, _vp, i64, _vp, i32, ctypes.POINTER(EchoCacheStruct), _vp, _vp,
                                               _vp, _vp, _vp, i32]
        L.echo_prefill_scores.restype = i32
        L.echo_prefill_scores.argtypes = [i32, i64, i64, _vp, _vp, _vp, _vp, _vp, i64, _vp, _vp, _vp, _vp]
        L.echo_prefill_workspace_size.restype = ctypes.c_size_t
        L.echo_prefill_workspace_size.argtypes = [i32, i64]
        L.echo_prefill_block.restype = i32
        L.echo_prefill_block.argtypes = [i32, i64, i64, _vp, _vp, _vp, _vp, i32, _vp, f32, _vp, i64, _vp, _vp,
                                         _vp, _vp, _vp, _vp, ctypes.POINTER(EchoCacheStruct), _vp, _vp,
                                         ctypes.c_size_t, _vp, _vp, _vp, _vp]
        L.echo_prefill_block_static.restype = i32
        L.echo_prefill_block_static.argtypes = [i32, i64, i64, _vp, _vp, _vp, _vp, i32, _vp, f32, _vp, i64, _vp,
                                                _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(EchoCacheStruct), _vp, _vp,
                                                _vp, _vp, _vp]
        L.echo_host_device_alias.restype = i32
        L.echo_host_device_alias.argtypes = [_vp, ctypes.POINTER(_vp)]
        L.echo_debug_stall_epilogue.restype = i32
        L.echo_debug_stall_epilogue.argtypes = [i64]
        L.echo_debug_wait_limit.restype = i32
        L.echo_debug_wait_limit.argtypes = [i64]
        L.echo_device_sm_count.restype = i32
        L.echo_device_sm_count.argtypes = []
        _lib = L
        return L


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _device():
    # torch.cuda.current_device() without its look at the initialisation (0.6 us a call)
    return torch.cuda.current_device() if _raw_stream is None or _raw_device is None else _raw_device()


def _stream(s):
    if s is None:
        if _raw_stream is not None:  # the same handle as below, without making a Stream object (3 us a call)
            return _raw_stream(_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(call, rc):
    if rc != ECHO_OK:
        raise EchoError(call, rc)


def host_device_alias(host_tensor: torch.Tensor) -> int:
    out = _vp()
    _check("echo_host_device_alias", load().echo_host_device_alias(host_tensor.data_ptr(), ctypes.byref(out)))
    return out.value


class _CudaArray:
    def __init__(self, iface):
        self.__cuda_array_interface__ = iface


_TYPESTR = {torch.int32: "<i4", torch.float32: "<f4", torch.uint8: "|u1", torch.int64: "<i8"}


def host_alias_tensor(host: torch.Tensor, device) -> torch.Tensor:
    """A CUDA tensor over the device alias of a pinned, contiguous host tensor (kernels
    read and write the host memory directly).  The caller keeps `host` alive."""
    if host.device.type != "cpu" or not host.is_pinned() or not host.is_contiguous():
        raise ValueError("host_alias_tensor needs a pinned, contiguous CPU tensor")
    iface = {"shape": tuple(host.shape), "typestr": _TYPESTR[host.dtype],
             "data": (host_device_alias(host), False), "version": 2, "strides": None}
    with torch.cuda.device(device):
        return torch.as_tensor(_CudaArray(iface), device=device)


def debug_stall_epilogue(limit_ns: int) -> None:
    """echo_debug_stall_epilogue: >= 0, every score call first waits on a barrier nothing arrives
    on and gives up after limit_ns (tests of the timeout path); < 0 turns that off."""
    _check("echo_debug_stall_epilogue", load().echo_debug_stall_epilogue(int(limit_ns)))


def debug_wait_limit(limit_ns: int) -> None:
    """echo_debug_wait_limit: the limit of the waits of later mla_chunk and mla_mass calls, from the last
    progress (< 0: the default, 2 s)."""
    _check("echo_debug_wait_limit", load().echo_debug_wait_limit(int(limit_ns)))


def sm_count() -> int:
    return load().echo_device_sm_count()


def quantize_q(q, w, q8, qscale, wfold, status, hist=None, stream=None, cand_cnt=None):
    """echo_quantize_q; q and w may be pinned host tensors, read by the kernel through their
    device alias; cand_cnt: the counts of a Cands (cleared with the histogram)."""
    B = q.shape[0]
    qp = host_device_alias(q) if q.device.type == "cpu" else _ptr(q)
    wp = host_device_alias(w) if w.device.type == "cpu" else _ptr(w)
    _check("echo_quantize_q", load().echo_quantize_q(B, qp, wp, _ptr(q8), _ptr(qscale),
                                                    _ptr(wfold), _ptr(hist), _ptr(cand_cnt), _ptr(status),
                                                    _stream(stream)))


def above_words(B: int, n_tokens: int) -> int:
    return int(load().echo_above_words(int(B), int(n_tokens)))


def index_scores(tok_off, n_tokens, q8, wfold, k8, ks, scores, theta_hat, hist, status, above=None,
                 cache=None, stream=None, ctas=0, tok_end=None, cands=None):
    """echo_index_scores; cache: a LayerCache whose residents `above` leaves out (and whose free bits
    are snapshotted for early_fetch); tok_end: the requests' current ends (None: full regions);
    cands: a Cands (or a view of one) to fill: echo_index_scores_cands."""
    B = q8.shape[0]
    cs = ctypes.byref(cache.struct) if cache is not None else None
    if cands is not None:
        _check("echo_index_scores_cands", load().echo_index_scores_cands(
            B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(q8), _ptr(wfold), _ptr(k8), _ptr(ks), _ptr(scores),
            _ptr(theta_hat), _ptr(hist), _ptr(above), cs, ctypes.byref(cands.struct), int(ctas), _ptr(status),
            _stream(stream)))
        return
    _check("echo_index_scores", load().echo_index_scores(
        B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(q8), _ptr(wfold), _ptr(k8), _ptr(ks), _ptr(scores),
        _ptr(theta_hat), _ptr(hist), _ptr(above), cs, int(ctas), _ptr(status), _stream(stream)))


def topk_select_cands(tok_off, n_tokens, scores, k, hist, theta_hat, alpha, cands, sel_idx, kth, status, stats=None,
                      stream=None, cache=None, sel_slot=None, above=None, early_cap=-1, tok_end=None):
    """echo_topk_select_cands: top-k from the candidate lists of `cands` (None: from all the
    scores), one block per request; with cache (and sel_slot) the cached form (slots of the
    selected tokens as echo_topk_select_cached gives them)."""
    B = tok_off.shape[0] - 1
    _check("echo_topk_select_cands", load().echo_topk_select_cands(
        B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(scores), int(k), _ptr(hist), _ptr(theta_hat),
        float(alpha), ctypes.byref(cands.struct) if cands is not None else None, _ptr(sel_idx), _ptr(kth),
        _ptr(above), int(early_cap), ctypes.byref(cache.struct) if cache is not None else None, _ptr(sel_slot),
        _ptr(status), _ptr(stats), _stream(stream)))


def early_fetch(tok_off, n_tokens, above, early_cap, cache, status, stream=None, tok_end=None):
    """echo_early_fetch: copy the rows of the early set (the tables learn it in cache_step)."""
    B = tok_off.shape[0] - 1
    _check("echo_early_fetch", load().echo_early_fetch(
        B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(above), int(early_cap), ctypes.byref(cache.struct), _ptr(status),
        _stream(stream)))


def topk_select(tok_off, n_tokens, scores, k, hist, theta_hat, alpha, sel_idx, kth, status, stats=None,
                stream=None, tok_end=None):
    B = tok_off.shape[0] - 1
    _check("echo_topk_select", load().echo_topk_select(
        B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(scores), int(k), _ptr(hist), _ptr(theta_hat), float(alpha),
        _ptr(sel_idx), _ptr(kth), _ptr(status), _ptr(stats), _stream(stream)))


def cache_step(tok_off, n_tokens, sel, cache, sel_slot, status, stats=None, stream=None, copy_stream=None,
               above=None, early_cap=-1, hold_early=False, tok_end=None, lazy=False):
    """echo_cache_step; above/early_cap: the early set of this step (as given to early_fetch);
    hold_early: ECHO_CACHE_HOLD_EARLY; lazy: ECHO_CACHE_LAZY (lazy-reuse eviction)."""
    B = tok_off.shape[0] - 1
    m = sel.shape[-1]
    st = _stream(stream)
    cst = _stream(copy_stream) if copy_stream is not None else st
    _check("echo_cache_step", load().echo_cache_step(
        B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(sel), int(m), _ptr(above), int(early_cap),
        ctypes.byref(cache.struct), _ptr(sel_slot), _ptr(status), _ptr(stats), st, cst,
        (CACHE_HOLD_EARLY if hold_early else 0) | (CACHE_LAZY if lazy else 0)))


def topk_select_cached(tok_off, n_tokens, scores, k, hist, theta_hat, alpha, sel_idx, kth, cache, sel_slot,
                       status, stats=None, stream=None, above=None, early_cap=-1, tok_end=None):
    """echo_topk_select_cached: top-k plus each selected token's slot at the cache step's start
    (resident or early; -1: a miss); finish with cache_step_resolved."""
    B = tok_off.shape[0] - 1
    _check("echo_topk_select_cached", load().echo_topk_select_cached(
        B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(scores), int(k), _ptr(hist), _ptr(theta_hat), float(alpha),
        _ptr(sel_idx), _ptr(kth), _ptr(above), int(early_cap), ctypes.byref(cache.struct), _ptr(sel_slot),
        _ptr(status), _ptr(stats), _stream(stream)))


def cache_step_resolved(tok_off, n_tokens, sel, cache, sel_slot, status, stats=None, stream=None, copy_stream=None,
                        hold_early=False, tok_end=None):
    """echo_cache_step_resolved: the cache step after topk_select_cached (sel_slot in/out)."""
    B = tok_off.shape[0] - 1
    m = sel.shape[-1]
    st = _stream(stream)
    cst = _stream(copy_stream) if copy_stream is not None else st
    _check("echo_cache_step_resolved", load().echo_cache_step_resolved(
        B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(sel), int(m), ctypes.byref(cache.struct), _ptr(sel_slot),
        _ptr(status), _ptr(stats), st, cst, CACHE_HOLD_EARLY if hold_early else 0))


def pool_above(tok_off, n_tokens, above_req, pool, above_pool, status, stream=None, tok_end=None):
    """echo_pool_above: per-request above words -> the shared pool's global marks (residents left
    out) and the pool's free-bit snapshot."""
    B = tok_off.shape[0] - 1
    _check("echo_pool_above", load().echo_pool_above(
        B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(above_req), ctypes.byref(pool.struct),
        _ptr(above_pool), _ptr(status), _stream(stream)))


def pool_select(tok_off, sel, sel_pool, stream=None):
    """echo_pool_select: sel [B,k] (request-local) -> sel_pool [B*k] (global, ascending, padding last)."""
    B, k = sel.shape
    _check("echo_pool_select", load().echo_pool_select(B, _ptr(tok_off), _ptr(sel), int(k), _ptr(sel_pool),
                                                       _stream(stream)))


def pool_slots(sel, slot_pool, sel_slot, stream=None):
    """echo_pool_slots: the pool step's slots of sel_pool -> sel_slot [B,k] aligned with sel."""
    B, k = sel.shape
    _check("echo_pool_slots", load().echo_pool_slots(B, _ptr(sel), int(k), _ptr(slot_pool), _ptr(sel_slot),
                                                     _stream(stream)))


def seed_early(tok_off, n_tokens, prev_sel, above, cache, status, stream=None, tok_end=None):
    """echo_seed_early: this layer's early set from the previous layer's selection prev_sel [B,m]
    (above words + cache free-bit snapshot); follow with early_fetch on the same above words."""
    B = tok_off.shape[0] - 1
    _check("echo_seed_early", load().echo_seed_early(
        B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(prev_sel), int(prev_sel.shape[-1]), _ptr(above),
        ctypes.byref(cache.struct), _ptr(status), _stream(stream)))


def append_tokens(tok_off, tok_end, n_tokens, k_new, kv_new, k8, ks, cache, status, stream=None):
    """echo_append_tokens: one new token per request (k_new [B,128] f32, kv_new [B,576] bf16, device)
    into its region at tok_end[b] (updated): E4M3 key + scale, host-pool row, and the lowest free
    cache slot when one is free."""
    B = tok_off.shape[0] - 1
    _check("echo_append_tokens", load().echo_append_tokens(
        B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(k_new), _ptr(kv_new), _ptr(k8), _ptr(ks),
        ctypes.byref(cache.struct), _ptr(status), _stream(stream)))


MLA_HEADS, MLA_DQK, MLA_DV, MLA_MAX_K = 128, 576, 512, 8192


def mla_decode(q, sel_slot, dev_kv, C, scale, out, lse, status, stream=None):
    """echo_mla_decode: q [B,128,576] bf16, sel_slot [B,k] int32, dev_kv [B*C,576] bf16 (the
    cache's rows) -> out [B,128,512] f32, lse [B,128] f32."""
    B, k = sel_slot.shape
    _check("echo_mla_decode", load().echo_mla_decode(
        int(B), int(k), _ptr(q), _ptr(sel_slot), _ptr(dev_kv), int(C), float(scale), _ptr(out), _ptr(lse),
        _ptr(status), _stream(stream)))


def _expect(call, dev, *tensors):
    # the layouts the C ABI takes: contiguous tensors of the given type and shape, on the current device
    for name, t, dtype, shape in tensors:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{call}: {name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the current "
                             f"CUDA device, not {t.dtype} {tuple(t.shape)} on {t.device}")


class KVPages:
    """A paged latent cache for mla_chunk / mla_mass (an echo_pages): token row g of the requests
    (tok_off) is cache row page_tab[g // page] * page + g % page of kv [rows, 576] bf16 (< 0: no
    row).  req_rows > 0: each request has that many kv rows of its own and its pages count from
    there.  Keeps the tensors alive; the table may change between calls, in place."""

    def __init__(self, page_tab: torch.Tensor, kv: torch.Tensor, page: int, req_rows: int = 0):
        if not 1 <= page < 2 ** 31 or not 0 <= req_rows < 2 ** 63:  # what the struct's fields hold
            raise ValueError("KVPages: 1 <= page < 2^31 and 0 <= req_rows < 2^63")
        _expect("KVPages", torch.cuda.current_device(), ("page_tab", page_tab, torch.int32, (page_tab.numel(),)),
                ("kv", kv, torch.bfloat16, (kv.shape[0], MLA_DQK)))
        self.page_tab, self.kv, self.page, self.req_rows = page_tab, kv, int(page), int(req_rows)
        self.tokens = page_tab.numel() * self.page
        s = EchoPagesStruct()
        s.page_tab, s.kv, s.kv_rows = _ptr(page_tab), _ptr(kv), kv.shape[0]
        s.req_rows, s.page, s.reserved = self.req_rows, self.page, 0
        self.struct = s

    @classmethod
    def of_cache(cls, cache: "LayerCache") -> "KVPages":
        """The slots of a LayerCache as pages of one row (a token that is not resident has no row; under lazy
        reuse one that was freed has its row until its slot is handed out)."""
        return cls(cache.tok2slot, cache.dev_kv, 1, cache.C)


def mla_chunk_workspace_size(n_rows: int, heads: int, B: int) -> int:
    return int(load().echo_mla_chunk_workspace_size(int(n_rows), int(heads), int(B)))


def _check_chunk(call, row_off, q, tok_off, n_tokens, pages, lse, status, tok_end, *more):
    if q.dim() != 3:
        raise ValueError(f"{call}: q must be a tensor of shape [rows, heads, {MLA_DQK}], not {tuple(q.shape)}")
    (n, heads, _), B, dev = q.shape, tok_off.shape[0] - 1, _device()
    _expect(call, dev, ("row_off", row_off, torch.int64, (B + 1,)), ("tok_off", tok_off, torch.int64, (B + 1,)),
            ("q", q, torch.bfloat16, (n, heads, MLA_DQK)), ("lse", lse, torch.float32, (n, heads)),
            ("status", status, torch.int32, (1,)), *more)
    if tok_end is not None:
        _expect(call, dev, ("tok_end", tok_end, torch.int64, (B,)))
    if pages.tokens < n_tokens or pages.kv.get_device() != dev:
        raise ValueError(f"{call}: the page table covers {pages.tokens} token rows, not {n_tokens}, or lies on another "
                         "device")
    return B, n, heads


def mla_chunk(row_off, q, tok_off, n_tokens, pages, scale, out, lse, ws, status, tok_end=None, window=0, sinks=0,
              sel=None, stream=None):
    """echo_mla_chunk: attention of each request's new rows q [n,heads,576] bf16 (row_off [B+1], at
    the end of its context) over the cache `pages` (a KVPages): causal; window > 0: the last
    `window` tokens and the first `sinks`; sel [n,k] int32: the tokens listed for each row -> out
    [n,heads,512] bf16, lse [n,heads] f32.  ws: uint8, mla_chunk_workspace_size(n, heads, B)."""
    k, more = 0, [("out", out, torch.bfloat16, (*q.shape[:2], MLA_DV)),
                  ("ws", ws, torch.uint8, (ws.numel(),))]
    if sel is not None:
        k = sel.shape[-1]
        more.append(("sel", sel, torch.int32, (q.shape[0], k)))
    B, n, heads = _check_chunk("mla_chunk", row_off, q, tok_off, n_tokens, pages, lse, status, tok_end, *more)
    _check("echo_mla_chunk", load().echo_mla_chunk(
        B, _ptr(row_off), n, heads, _ptr(q), _ptr(tok_off), _ptr(tok_end), int(n_tokens),
        ctypes.byref(pages.struct), _ptr(sel), k, int(window), int(sinks), float(scale), _ptr(out), _ptr(lse),
        _ptr(ws), ws.numel(), _ptr(status), _stream(stream)))


def mla_mass_workspace_size(n_tokens: int, B: int) -> int:
    return int(load().echo_mla_mass_workspace_size(int(n_tokens), int(B)))


def mla_mass(row_off, q, lse, tok_off, n_tokens, pages, scale, mass, mass_out, status, decay=1.0, tok_end=None,
             window=0, sinks=0, ws=None, stream=None):
    """echo_mla_mass: mass_out [n_tokens] f32 = decay * mass + the attention weight each token
    receives from the rows of an mla_chunk call (the same q, pages, window and sinks, and its lse),
    summed over rows and heads.  mass_out may be mass.  ws: uint8, mla_mass_workspace_size(n_tokens,
    B) (None: one is taken from torch's allocator, on `stream`, for the call)."""
    B, n, heads = _check_chunk("mla_mass", row_off, q, tok_off, n_tokens, pages, lse, status, tok_end,
                               ("mass", mass, torch.float32, (n_tokens,)),
                               ("mass_out", mass_out, torch.float32, (n_tokens,)))
    if ws is None:
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            raise ValueError("mla_mass: a stream given by its handle needs ws")
        # from the pool of the stream that uses it: a block of the current stream's pool may still be read or
        # written by kernels pending there when it is handed out
        with torch.cuda.stream(stream):
            ws = torch.empty(mla_mass_workspace_size(n_tokens, B), dtype=torch.uint8, device=q.device)
    else:
        _expect("mla_mass", torch.cuda.current_device(), ("ws", ws, torch.uint8, (ws.numel(),)))
    _check("echo_mla_mass", load().echo_mla_mass(
        B, _ptr(row_off), n, heads, _ptr(q), _ptr(lse), _ptr(tok_off), _ptr(tok_end), int(n_tokens),
        ctypes.byref(pages.struct), int(window), int(sinks), float(scale), _ptr(mass), _ptr(mass_out), float(decay),
        _ptr(ws), ws.numel(), _ptr(status), _stream(stream)))


def tree_masks(row_off, parent, mask, status, depth=None, stream=None):
    """echo_tree_masks: the ancestors of every node of the requests' draft trees.  parent [n] int32 (request-local,
    -1: none) -> mask [n,words] int32, a bit for each node of the request, depth [n] int32 (or None)."""
    B, n, words = row_off.shape[0] - 1, parent.shape[0], mask.shape[-1]
    _expect("tree_masks", _device(), ("row_off", row_off, torch.int64, (B + 1,)), ("parent", parent, torch.int32, (n,)),
            ("mask", mask, torch.int32, (n, words)), ("status", status, torch.int32, (1,)),
            *([] if depth is None else [("depth", depth, torch.int32, (n,))]))
    _check("echo_tree_masks", load().echo_tree_masks(B, row_off.data_ptr(), n, parent.data_ptr(), words, mask.data_ptr(),
                                                     _ptr(depth), status.data_ptr(), _stream(stream)))


def mla_tree(row_off, q, mask, tok_off, n_tokens, pages, scale, out, lse, ws, status, tok_end=None, stream=None):
    """echo_mla_tree: mla_chunk where a request's new rows are the nodes of a draft tree: each sees the whole context
    before the tree and, of the tree, the nodes up to itself whose bit its row of mask [n,words] int32 has
    (tree_masks).  ws as mla_chunk's."""
    words = mask.shape[-1]
    B, n, heads = _check_chunk("mla_tree", row_off, q, tok_off, n_tokens, pages, lse, status, tok_end,
                               ("out", out, torch.bfloat16, (*q.shape[:2], MLA_DV)),
                               ("mask", mask, torch.int32, (q.shape[0], words)), ("ws", ws, torch.uint8, (ws.numel(),)))
    _check("echo_mla_tree", load().echo_mla_tree(
        B, row_off.data_ptr(), n, heads, q.data_ptr(), mask.data_ptr(), words, tok_off.data_ptr(), _ptr(tok_end),
        int(n_tokens), pages.struct, float(scale), out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
        status.data_ptr(), _stream(stream)))


def draft_verify(row_off, parent, token, target, path, count, next_tok, status, draft=None, u_node=None, u_pick=None,
                 stream=None):
    """echo_draft_verify: the path of each request's draft tree that the target accepts, and the token behind it.
    parent, token [n] int32; target [n,vocab] f32 or bf16: the target's probabilities behind each node; draft [n,vocab]
    of the same type: those its children were drawn from (None: drafts without probabilities); u_node [n] and u_pick [B]
    f32: uniform numbers in [0, 1) (both None: greedy, target may hold logits) -> path [n] int32 (accepted nodes from
    row_off[b] on, -1 behind), count [B] int32, next_tok [B] int32."""
    if target.dim() != 2:
        raise ValueError(f"draft_verify: target must be a tensor of shape [rows, vocab], not {tuple(target.shape)}")
    B, (n, vocab), dtype = row_off.shape[0] - 1, target.shape, target.dtype
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"draft_verify: target must be float32 or bfloat16, not {dtype}")
    if (u_node is None) != (u_pick is None):
        raise ValueError("draft_verify: u_node and u_pick go together")
    _expect("draft_verify", _device(), ("row_off", row_off, torch.int64, (B + 1,)), ("parent", parent, torch.int32, (n,)),
            ("token", token, torch.int32, (n,)), ("target", target, dtype, (n, vocab)), ("path", path, torch.int32, (n,)),
            ("count", count, torch.int32, (B,)), ("next_tok", next_tok, torch.int32, (B,)),
            ("status", status, torch.int32, (1,)), *([] if draft is None else [("draft", draft, dtype, (n, vocab))]),
            *([] if u_node is None else [("u_node", u_node, torch.float32, (n,)), ("u_pick", u_pick, torch.float32, (B,))]))
    _check("echo_draft_verify", load().echo_draft_verify(
        B, row_off.data_ptr(), n, parent.data_ptr(), token.data_ptr(), vocab,
        DTYPE_F32 if dtype is torch.float32 else DTYPE_BF16, target.data_ptr(), _ptr(draft), _ptr(u_node), _ptr(u_pick),
        path.data_ptr(), count.data_ptr(), next_tok.data_ptr(), status.data_ptr(), _stream(stream)))


class PagePool:
    """The pages of a paged cache with the counts of who holds them (an echo_page_pool): page_tab [entries] int32 (as
    KVPages'; -1: no page), refs [n_pages] int32 (0: free), kv [n_pages * page, 576] bf16, or [layers, n_pages * page, 576]
    with one table for every layer.  An empty pool has page_tab all -1 and refs all 0.  Keeps the tensors alive."""

    def __init__(self, page_tab: torch.Tensor, refs: torch.Tensor, kv: torch.Tensor, page: int):
        if not 1 <= page < 2 ** 31:
            raise ValueError("PagePool: 1 <= page < 2^31")
        n = refs.numel()
        shape = (n * page, MLA_DQK) if kv.dim() == 2 else (kv.shape[0], n * page, MLA_DQK)
        _expect("PagePool", _device(), ("page_tab", page_tab, torch.int32, (page_tab.numel(),)),
                ("refs", refs, torch.int32, (n,)), ("kv", kv, torch.bfloat16, shape))
        self.page_tab, self.refs, self.kv, self.page, self.n_pages = page_tab, refs, kv, int(page), n
        self.layers = 1 if kv.dim() == 2 else kv.shape[0]
        self.tokens, self.device = page_tab.numel() * self.page, kv.get_device()
        s = EchoPagePoolStruct()
        s.page_tab, s.refs, s.kv, s.n_pages = _ptr(page_tab), _ptr(refs), _ptr(kv), n
        s.row_bytes, s.layer_bytes, s.layers, s.page = 2 * MLA_DQK, 2 * MLA_DQK * n * self.page, self.layers, self.page
        self.struct = s

    def of_layer(self, layer: int = 0) -> "KVPages":
        """The pages of a layer, for mla_chunk, mla_mass and mla_tree."""
        return KVPages(self.page_tab, self.kv if self.kv.dim() == 2 else self.kv[layer], self.page)


def pages_workspace_size(B: int, n_pages: int) -> int:
    return int(load().echo_pages_workspace_size(int(B), int(n_pages)))


def _check_table(call, n_tokens, pool, dev):
    if pool.tokens < n_tokens or pool.device != dev:
        raise ValueError(f"{call}: the page table covers {pool.tokens} token rows, not {n_tokens}, or lies on another device")


def pages_reserve(tok_off, tok_end, want, n_tokens, pool, room, ws, status, stream=None):
    """echo_pages_reserve: pages for the tokens [tok_end[b], want[b]) of every request (want [B] int64, token rows),
    the lowest free ones; a page others hold too is replaced.  room [B] int64 (or None): want[b] where served, else
    tok_end[b].  ws: uint8, pages_workspace_size(B, n_pages)."""
    B, dev, i64 = tok_off.shape[0] - 1, _device(), torch.int64
    per = (B,)
    _expect("pages_reserve", dev, ("tok_off", tok_off, i64, (B + 1,)), ("status", status, torch.int32, (1,)),
            ("tok_end", tok_end, i64, per), ("want", want, i64, per), ("ws", ws, torch.uint8, (ws.numel(),)),
            *(() if room is None else (("room", room, i64, per),)))
    _check_table("pages_reserve", n_tokens, pool, dev)
    _check("echo_pages_reserve", load().echo_pages_reserve(
        B, tok_off.data_ptr(), tok_end.data_ptr(), want.data_ptr(), int(n_tokens), pool.struct, _ptr(room), ws.data_ptr(),
        ws.numel(), status.data_ptr(), _stream(stream)))


def pages_free(tok_off, tok_end, n_tokens, pool, status, stream=None):
    """echo_pages_free: gives up the pages behind every request's end (tok_end[b] = tok_off[b]: all of them)."""
    B, dev = tok_off.shape[0] - 1, _device()
    _expect("pages_free", dev, ("tok_off", tok_off, torch.int64, (B + 1,)), ("status", status, torch.int32, (1,)),
            ("tok_end", tok_end, torch.int64, (B,)))
    _check_table("pages_free", n_tokens, pool, dev)
    _check("echo_pages_free", load().echo_pages_free(B, tok_off.data_ptr(), tok_end.data_ptr(), int(n_tokens), pool.struct,
                                                     status.data_ptr(), _stream(stream)))


def pages_fork(src, dst, tok_off, tok_end, n_tokens, pool, ws, status, stream=None):
    """echo_pages_fork: request dst[i] gives up its pages and gets the context of request src[i] (src, dst [m] int32):
    full pages shared, the rows of a partly used last page copied, tok_end[dst[i]] set.  ws: uint8,
    pages_workspace_size(m, n_pages)."""
    m, B, dev = src.numel(), tok_off.shape[0] - 1, _device()
    _expect("pages_fork", dev, ("tok_off", tok_off, torch.int64, (B + 1,)), ("status", status, torch.int32, (1,)),
            ("tok_end", tok_end, torch.int64, (B,)), ("src", src, torch.int32, (m,)), ("dst", dst, torch.int32, (m,)),
            ("ws", ws, torch.uint8, (ws.numel(),)))
    _check_table("pages_fork", n_tokens, pool, dev)
    _check("echo_pages_fork", load().echo_pages_fork(
        m, src.data_ptr(), dst.data_ptr(), B, tok_off.data_ptr(), tok_end.data_ptr(), int(n_tokens), pool.struct,
        ws.data_ptr(), ws.numel(), status.data_ptr(), _stream(stream)))


def pages_compact(n_tokens, pool, used, ws, status, stream=None):
    """echo_pages_compact: the pages in use move to the first places of the pool, their rows, counts and table entries
    with them; used [1] int32: how many there are.  ws: uint8, pages_workspace_size(1, n_pages)."""
    dev = _device()
    _expect("pages_compact", dev, ("used", used, torch.int32, (1,)), ("ws", ws, torch.uint8, (ws.numel(),)),
            ("status", status, torch.int32, (1,)))
    _check_table("pages_compact", n_tokens, pool, dev)
    _check("echo_pages_compact", load().echo_pages_compact(int(n_tokens), pool.struct, used.data_ptr(), ws.data_ptr(),
                                                           ws.numel(), status.data_ptr(), _stream(stream)))


def rows_keep(row_off, path, count, tok_off, tok_end, n_tokens, pool, new_end, status, stream=None):
    """echo_rows_keep: the cache rows of the accepted nodes of each request's draft tree (path, count of
    draft_verify) move together behind the context, in every layer; new_end [B] int64: where the contexts then end
    (not tok_end itself).  pages_free(new_end) gives up the pages behind."""
    B, n, dev, i64, i32 = tok_off.shape[0] - 1, path.numel(), _device(), torch.int64, torch.int32
    ends, per = (B + 1,), (B,)
    _expect("rows_keep", dev, ("tok_off", tok_off, i64, ends), ("status", status, i32, (1,)), ("tok_end", tok_end, i64, per),
            ("new_end", new_end, i64, per), ("row_off", row_off, i64, ends), ("path", path, i32, (n,)), ("count", count, i32, per))
    _check_table("rows_keep", n_tokens, pool, dev)
    _check("echo_rows_keep", load().echo_rows_keep(
        B, row_off.data_ptr(), n, path.data_ptr(), count.data_ptr(), tok_off.data_ptr(), tok_end.data_ptr(), int(n_tokens),
        pool.struct, new_end.data_ptr(), status.data_ptr(), _stream(stream)))


def evict_select(tok_off, n_tokens, slot2tok, mass, keep, evict_tok, evict_slot, evict_cnt, status, sinks=0, recent=0,
                 tok_end=None, stream=None, freebits=None):
    """echo_evict_select: the victims of each request's cache (slot2tok [B*C] or [B,C]) when it has to
    shrink to `keep` residents: those of the lowest mass [n_tokens], the first `sinks` and last
    `recent` tokens spared -> evict_tok / evict_slot [B,C] (ascending slots, -1 behind), evict_cnt [B].
    freebits: the cache's free bits (a LayerCache's, or a slice of them); a cache under lazy reuse needs them, as
    its free slots keep their tokens."""
    B = tok_off.shape[0] - 1
    C = slot2tok.numel() // max(B, 1)
    dev = torch.cuda.current_device()
    _expect("evict_select", dev, ("tok_off", tok_off, torch.int64, (B + 1,)),
            ("slot2tok", slot2tok, torch.int32, (B * C,) if slot2tok.dim() == 1 else (B, C)),
            ("mass", mass, torch.float32, (n_tokens,)), ("evict_tok", evict_tok, torch.int32, (B, C)),
            ("evict_slot", evict_slot, torch.int32, (B, C)), ("evict_cnt", evict_cnt, torch.int32, (B,)),
            ("status", status, torch.int32, (1,)))
    if tok_end is not None:
        _expect("evict_select", dev, ("tok_end", tok_end, torch.int64, (B,)))
    if freebits is not None:
        _expect("evict_select", dev, ("freebits", freebits, torch.int32, (B * C // 32,)))
    _check("echo_evict_select_resident", load().echo_evict_select_resident(
        B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(slot2tok), _ptr(freebits), C, _ptr(mass), int(keep),
        int(sinks), int(recent), _ptr(evict_tok), _ptr(evict_slot), _ptr(evict_cnt), _ptr(status), _stream(stream)))


def cache_release(tok_off, n_tokens, tok, cache, status, mass=None, tok_end=None, stream=None):
    """echo_cache_release: frees the slots of the listed tokens (tok [B,m] int32, -1 padding) that are
    resident in `cache`; with mass [n_tokens], their masses become 0."""
    B = tok_off.shape[0] - 1
    m = tok.shape[-1]
    dev = torch.cuda.current_device()
    _expect("cache_release", dev, ("tok_off", tok_off, torch.int64, (B + 1,)), ("tok", tok, torch.int32, (B, m)),
            ("status", status, torch.int32, (1,)))
    if tok_end is not None:
        _expect("cache_release", dev, ("tok_end", tok_end, torch.int64, (B,)))
    if mass is not None:
        _expect("cache_release", dev, ("mass", mass, torch.float32, (n_tokens,)))
    whole = getattr(cache, "parent", cache)             # of a CacheView
    requests = cache.B if whole is cache else cache.b1 - cache.b0
    if whole.n_tokens < n_tokens or requests != B or whole.tok2slot.get_device() != dev:
        raise ValueError(f"cache_release: a cache of {requests} requests and {whole.n_tokens} token rows, not {B} and "
                         f"{n_tokens}, or on another device")
    _check("echo_cache_release", load().echo_cache_release(
        B, _ptr(tok_off), _ptr(tok_end), int(n_tokens), _ptr(tok), m, ctypes.byref(cache.struct), _ptr(mass),
        _ptr(status), _stream(stream)))


def prefill_scores(R, row0, n_keys, q8, wfold, k8, ks, scores, W, theta_hat, hist, status, stream=None):
    _check("echo_prefill_scores", load().echo_prefill_scores(
        int(R), int(row0), int(n_keys), _ptr(q8), _ptr(wfold), _ptr(k8), _ptr(ks), _ptr(scores), int(W),
        _ptr(theta_hat), _ptr(hist), _ptr(status), _stream(stream)))


def prefill_workspace_size(R: int, W: int) -> int:
    return int(load().echo_prefill_workspace_size(int(R), int(W)))


def prefill_block(R, row0, n_keys, q, w, k8, ks, k, theta_hat, alpha, scores, W, hist, sel_idx, kth,
                  union_list, union_count, union_bits, cache, sel_slot, ws, status, stats=None, stream=None,
                  copy_stream=None):
    st = _stream(stream)
    cst = _stream(copy_stream) if copy_stream is not None else st
    _check("echo_prefill_block", load().echo_prefill_block(
        int(R), int(row0), int(n_keys), _ptr(q), _ptr(w), _ptr(k8), _ptr(ks), int(k), _ptr(theta_hat),
        float(alpha), _ptr(scores), int(W), _ptr(hist), _ptr(sel_idx), _ptr(kth), _ptr(union_list),
        _ptr(union_count), _ptr(union_bits), ctypes.byref(cache.struct) if cache is not None else None,
        _ptr(sel_slot), _ptr(ws), ws.numel() * ws.element_size(), _ptr(status), _ptr(stats), st, cst))


def prefill_block_static(R, row0, n_keys, q, w, k8, ks, k, theta_hat, alpha, scores, W, hist, sel_idx, kth,
                         union_list, union_count, union_bits, cache, sel_slot, status, stats=None, stream=None,
                         copy_stream=None):
    """echo_prefill_block with the library's fixed device scratch instead of a workspace."""
    st = _stream(stream)
    cst = _stream(copy_stream) if copy_stream is not None else st
    _check("echo_prefill_block_static", load().echo_prefill_block_static(
        int(R), int(row0), int(n_keys), _ptr(q), _ptr(w), _ptr(k8), _ptr(ks), int(k), _ptr(theta_hat),
        float(alpha), _ptr(scores), int(W), _ptr(hist), _ptr(sel_idx), _ptr(kth), _ptr(union_list),
        _ptr(union_count), _ptr(union_bits), ctypes.byref(cache.struct) if cache is not None else None,
        _ptr(sel_slot), _ptr(status), _ptr(stats), st, cst))


class Cands:
    """Candidate lists of decode top-k for B requests (torch-owned, int32 storage): key / idx
    [B*cap], cnt [B] (cleared by quantize_q when passed as cand_cnt), cut [B] (all ones = no
    list yet; top-k writes the next step's)."""

    def __init__(self, B: int, cap: int = CAND_CAP, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.B, self.cap, self.b0 = int(B), int(cap), 0
        self.key = torch.zeros(max(self.B * self.cap, 1), **i32)
        self.idx = torch.zeros(max(self.B * self.cap, 1), **i32)
        self.cnt = torch.zeros(max(self.B, 1), **i32)
        self.cut = torch.full((max(self.B, 1),), -1, **i32)
        self.struct = self._struct(0)

    def _struct(self, b0: int) -> EchoCandsStruct:
        # b0: absolute first request in the storage of the lists this object was made from
        root = getattr(self, "_parent", self)
        s = EchoCandsStruct()
        s.key, s.idx = _ptr(root.key[b0 * self.cap:]), _ptr(root.idx[b0 * self.cap:])
        s.cnt, s.cut = _ptr(root.cnt[b0:]), _ptr(root.cut[b0:])
        s.cap, s.reserved = self.cap, 0
        return s

    def view(self, b0: int, b1: int) -> "Cands":
        """The lists of requests [b0, b1) of this object (shared storage)."""
        root = getattr(self, "_parent", self)
        a0, a1 = self.b0 + int(b0), self.b0 + int(b1)
        v = Cands.__new__(Cands)
        v._parent = root
        v.B, v.cap, v.b0 = a1 - a0, self.cap, a0
        v.key, v.idx = root.key, root.idx
        v.cnt, v.cut = root.cnt[a0:a1], root.cut[a0:a1]
        v.struct = v._struct(a0)
        return v

    def reset(self):
        self.cnt.zero_()
        self.cut.fill_(-1)


class LayerCache:
    """The fixed-size GPU cache tensors of one layer for B requests (torch-owned).

    host_pool: pinned host tensor [n_tokens, row_bytes/2] bf16 (the per-layer
    host copy of every token's KV row)."""

    def __init__(self, B: int, n_tokens: int, C: int, host_pool: torch.Tensor, device="cuda"):
        if C % 32:
            raise ValueError("C must be a multiple of 32")
        assert host_pool.is_pinned()
        self.B, self.C, self.n_tokens = B, C, n_tokens
        self.row_bytes = host_pool.shape[1] * host_pool.element_size()
        i32 = dict(dtype=torch.int32, device=device)
        self.tok2slot = torch.full((max(n_tokens, 1),), -1, **i32)
        self.slot2tok = torch.full((B * C,), -1, **i32)
        self.freebits = torch.full((B * C // 32,), -1, **i32)   # all bits set: every slot free
        self.miss_tok = torch.zeros((B * C,), **i32)
        self.miss_slot = torch.zeros((B * C,), **i32)
        self.miss_cnt = torch.zeros((B,), **i32)
        self.early_tok = torch.zeros((B * C,), **i32)
        self.early_slot = torch.zeros((B * C,), **i32)
        self.early_cnt = torch.zeros((B,), **i32)
        self.free_snap = torch.zeros((B * C // 32,), **i32)
        self.dev_kv = torch.zeros((B * C, host_pool.shape[1]), dtype=host_pool.dtype, device=device)
        self.host_pool = host_pool
        self.host_alias = host_device_alias(host_pool)
        s = EchoCacheStruct()
        s.tok2slot, s.slot2tok, s.freebits = _ptr(self.tok2slot), _ptr(self.slot2tok), _ptr(self.freebits)
        s.miss_tok, s.miss_slot, s.miss_cnt = _ptr(self.miss_tok), _ptr(self.miss_slot), _ptr(self.miss_cnt)
        s.early_tok, s.early_slot, s.early_cnt = (_ptr(self.early_tok), _ptr(self.early_slot),
                                                  _ptr(self.early_cnt))
        s.free_snap = _ptr(self.free_snap)
        s.host_kv, s.dev_kv = self.host_alias, _ptr(self.dev_kv)
        s.row_bytes, s.C, s.reserved = self.row_bytes, C, 0
        self.struct = s

    def view(self, b0: int, b1: int) -> "CacheView":
        """The tables of requests [b0, b1) as a cache of b1 - b0 requests (shared storage)."""
        return CacheView(self, b0, b1)

    def reset(self):
        self.tok2slot.fill_(-1)
        self.slot2tok.fill_(-1)
        self.freebits.fill_(-1)
        self.miss_cnt.zero_()
        self.early_cnt.zero_()


class CacheView:
    """Requests [b0, b1) of a LayerCache: per-request arrays offset to b0, tok2slot and the host
    pool shared (token rows are global).  Holds the parent so its storage stays alive."""

    def __init__(self, parent: LayerCache, b0: int, b1: int):
        self.parent, self.b0, self.b1 = parent, int(b0), int(b1)
        C, words = parent.C, parent.C // 32
        s = EchoCacheStruct()
        s.tok2slot = _ptr(parent.tok2slot)
        s.slot2tok = _ptr(parent.slot2tok[b0 * C:])
        s.freebits = _ptr(parent.freebits[b0 * words:])
        s.miss_tok, s.miss_slot = _ptr(parent.miss_tok[b0 * C:]), _ptr(parent.miss_slot[b0 * C:])
        s.miss_cnt = _ptr(parent.miss_cnt[b0:])
        s.early_tok, s.early_slot = _ptr(parent.early_tok[b0 * C:]), _ptr(parent.early_slot[b0 * C:])
        s.early_cnt = _ptr(parent.early_cnt[b0:])
        s.free_snap = _ptr(parent.free_snap[b0 * words:])
        s.host_kv, s.dev_kv = parent.host_alias, _ptr(parent.dev_kv[b0 * C:])
        s.row_bytes, s.C, s.reserved = parent.row_bytes, C, 0
        self.struct = s
