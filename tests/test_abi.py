"""The C-ABI library builds, loads and exports every entry point its header
declares; host-side argument checks answer without touching a GPU (CPU only)."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "echo.h")


def _declared():
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:[\w\s\*]+?)\b(echo_\w+)\s*\(", src, flags=re.M)))


@pytest.fixture(scope="module")
def L():
    from sparse_attention_kv_echo_gb300 import build, lib
    build.build()
    return lib.load()


def test_header_declares_the_calls():
    names = _declared()
    for want in ("echo_index_scores", "echo_topk_select", "echo_cache_step", "echo_quantize_q",
                 "echo_early_fetch", "echo_prefill_block"):
        assert want in names


def test_every_declared_symbol_is_exported(L):
    from sparse_attention_kv_echo_gb300 import build
    out = subprocess.run(["nm", "-D", "--defined-only", build.LIB], capture_output=True, text=True,
                         check=True).stdout
    exported = set(re.findall(r"\bT (echo_\w+)", out))
    for name in _declared():
        assert name in exported, name
        assert hasattr(L, name)


def test_binding_lists_every_export(L):
    from sparse_attention_kv_echo_gb300 import lib
    assert sorted(lib.EXPORTS) == _declared()


def test_host_checks_reject_bad_arguments(L):
    """These return before any CUDA call, so they run without a GPU."""
    from sparse_attention_kv_echo_gb300 import lib
    v = ctypes.c_void_p
    dummy = v(0x1000)
    # index_scores(B, tok_off, tok_end, n_tokens, q8, wfold, k8, ks, scores, theta, hist, above, cache, ctas,
    #              status, stream)
    def scores_call(B=1, n=10, q8=dummy, k8=dummy, above=None, cache=None):
        return L.echo_index_scores(B, dummy, None, n, q8, dummy, k8, dummy, dummy, None, None, above, cache, 0, dummy,
                                   None)
    assert scores_call(B=0) == lib.ECHO_EINVAL
    assert scores_call(B=lib.MAX_REQUESTS + 1) == lib.ECHO_EUNSUPPORTED
    assert scores_call(q8=None) == lib.ECHO_EINVAL                     # missing q8
    assert scores_call(k8=v(0x1001)) == lib.ECHO_EINVAL                # keys must be 16-byte aligned
    assert scores_call(n=-5) == lib.ECHO_EINVAL                        # negative token count
    assert scores_call(n=0) == lib.ECHO_OK                             # no tokens: nothing enqueued
    # a cache needs the above-threshold words, a complete struct and the snapshot
    c = lib.EchoCacheStruct()
    for f, _ in lib.EchoCacheStruct._fields_:
        if f not in ("row_bytes", "C", "reserved"):
            setattr(c, f, 0x1000)
    c.row_bytes, c.C = 1152, 64
    cache = ctypes.byref(c)
    assert scores_call(above=None, cache=cache) == lib.ECHO_EINVAL
    c.free_snap = None
    assert scores_call(above=dummy, cache=cache) == lib.ECHO_EINVAL
    # early_fetch(B, tok_off, tok_end, n_tokens, above, early_cap, cache, status, stream)
    assert L.echo_early_fetch(1, dummy, None, 10, dummy, -1, cache, dummy, None) == lib.ECHO_EINVAL   # no snapshot
    c.free_snap = 0x1000
    assert L.echo_early_fetch(1, dummy, None, 10, None, -1, cache, dummy, None) == lib.ECHO_EINVAL    # no above words
    assert L.echo_early_fetch(1, dummy, None, 10, dummy, -1, None, dummy, None) == lib.ECHO_EINVAL    # no cache
    assert L.echo_early_fetch(0, dummy, None, 10, dummy, -1, cache, dummy, None) == lib.ECHO_EINVAL
    assert L.echo_early_fetch(1, dummy, None, 0, dummy, -1, cache, dummy, None) == lib.ECHO_OK        # nothing to do
    assert L.echo_early_fetch(1, dummy, None, 10, dummy, 0, cache, dummy, None) == lib.ECHO_OK        # cap 0: nothing
    c.C = 48                                                           # not a multiple of 32
    assert L.echo_early_fetch(1, dummy, None, 10, dummy, -1, cache, dummy, None) == lib.ECHO_ECAPACITY
    assert scores_call(above=dummy, cache=cache) == lib.ECHO_ECAPACITY
    # the bitmask size: four words per 128-token tile of each request, at most
    assert lib.above_words(8, 32768) == 4 * (256 + 8)
    assert lib.above_words(0, 10) == 0
    assert L.echo_topk_select(1, dummy, None, 10, dummy, 0, None, None, 0.5, dummy, dummy, dummy, None,
                              None) == lib.ECHO_EINVAL
    assert L.echo_topk_select(-3, dummy, None, 10, dummy, 4, None, None, 0.5, dummy, dummy, dummy, None,
                              None) == lib.ECHO_EINVAL
    # quantize_q(B, q, w, q8, qscale, wfold, hist, cand_cnt, status, stream)
    assert L.echo_quantize_q(-1, dummy, dummy, dummy, dummy, dummy, None, None, dummy, None) == lib.ECHO_EINVAL
    assert L.echo_quantize_q(1, dummy, dummy, dummy, dummy, v(0x1004), None, None, dummy, None) == lib.ECHO_EINVAL
    assert L.echo_quantize_q(1, dummy, dummy, dummy, dummy, dummy, None, v(0x1002), dummy, None) == lib.ECHO_EINVAL
    assert L.echo_quantize_q(0, None, None, None, None, None, None, None, None, None) == lib.ECHO_OK


def test_candidate_list_checks(L):
    """echo_index_scores_cands needs complete lists; echo_topk_select_cands refuses bad sizes,
    incomplete lists and a cache without sel_slot or above its shared-memory limit."""
    from sparse_attention_kv_echo_gb300 import lib
    v = ctypes.c_void_p
    d = v(0x1000)
    cl = lib.EchoCandsStruct()
    cl.key, cl.idx, cl.cnt, cl.cut, cl.cap = 0x1000, 0x1000, 0x1000, 0x1000, 64
    cands = ctypes.byref(cl)

    def scores(c, n=10):
        return L.echo_index_scores_cands(1, d, None, n, d, d, d, d, d, None, None, None, None, c, 0, d, None)
    assert scores(None) == lib.ECHO_EINVAL
    assert scores(cands, n=0) == lib.ECHO_OK
    cl.cap = 0
    assert scores(cands) == lib.ECHO_EINVAL
    cl.cap, cl.cut = 64, None
    assert scores(cands) == lib.ECHO_EINVAL
    cl.cut = 0x1000

    # topk_select_cands(B, tok_off, tok_end, n, scores, k, hist, theta, alpha, cands, sel, kth, above, cap,
    #                   cache, sel_slot, status, stats, stream)
    def topk(B=1, k=16, c=cands, cache=None, slot=None):
        return L.echo_topk_select_cands(B, d, None, 100, d, k, None, None, 0.5, c, d, d, None, -1, cache, slot, d,
                                        None, None)
    assert topk(B=0) == lib.ECHO_EINVAL
    assert topk(k=0) == lib.ECHO_EINVAL
    assert topk(B=lib.MAX_REQUESTS + 1) == lib.ECHO_EUNSUPPORTED
    cl.idx = None
    assert topk() == lib.ECHO_EINVAL
    cl.idx = 0x1000
    s = lib.EchoCacheStruct()
    for f, _ in lib.EchoCacheStruct._fields_[:12]:
        setattr(s, f, 0x2000)
    s.row_bytes, s.C = 1152, 64
    assert topk(cache=ctypes.byref(s)) == lib.ECHO_EINVAL                    # no sel_slot
    assert topk(k=65, cache=ctypes.byref(s), slot=d) == lib.ECHO_ECAPACITY   # k > C
    s.C = 65536
    assert topk(cache=ctypes.byref(s), slot=d) == lib.ECHO_EUNSUPPORTED      # free bits beyond shared memory


def test_cache_checks(L):
    from sparse_attention_kv_echo_gb300 import lib
    v = ctypes.c_void_p
    s = lib.EchoCacheStruct()
    for f, _ in lib.EchoCacheStruct._fields_[:12]:
        setattr(s, f, 0x2000)
    s.row_bytes, s.C = 1152, 64
    dummy = v(0x1000)
    # k (m) larger than C
    assert L.echo_cache_step(1, dummy, None, 100, dummy, 65, None, 0, ctypes.byref(s), dummy, dummy, None, None,
                             None, 0) == lib.ECHO_ECAPACITY
    s.C = 48   # not a multiple of 32
    assert L.echo_cache_step(1, dummy, None, 100, dummy, 16, None, 0, ctypes.byref(s), dummy, dummy, None, None,
                             None, 0) == lib.ECHO_ECAPACITY
    s.C, s.row_bytes = 64, 1000  # row not a multiple of 16 bytes
    assert L.echo_cache_step(1, dummy, None, 100, dummy, 16, None, 0, ctypes.byref(s), dummy, dummy, None, None,
                             None, 0) == lib.ECHO_EUNSUPPORTED
    s.row_bytes, s.dev_kv = 1152, None
    assert L.echo_cache_step(1, dummy, None, 100, dummy, 16, None, 0, ctypes.byref(s), dummy, dummy, None, None,
                             None, 0) == lib.ECHO_EINVAL
    s.dev_kv = 0x2000
    # unknown flag bits; the held-slot form and lazy reuse together; lazy reuse in the resolved form
    assert L.echo_cache_step(1, dummy, None, 100, dummy, 16, None, 0, ctypes.byref(s), dummy, dummy, None, None,
                             None, 4) == lib.ECHO_EINVAL
    assert L.echo_cache_step(1, dummy, None, 100, dummy, 16, None, 0, ctypes.byref(s), dummy, dummy, None, None,
                             None, lib.CACHE_HOLD_EARLY | lib.CACHE_LAZY) == lib.ECHO_EINVAL
    assert L.echo_cache_step_resolved(1, dummy, None, 100, dummy, 16, ctypes.byref(s), dummy, dummy, None, None,
                                      None, lib.CACHE_LAZY) == lib.ECHO_EINVAL
    assert L.echo_cache_step_resolved(1, dummy, None, 100, dummy, 16, ctypes.byref(s), dummy, dummy, None, None,
                                      None, 4) == lib.ECHO_EINVAL
    # the resolved form: k larger than C; the cached top-k: C above its shared-memory limit
    assert L.echo_cache_step_resolved(1, dummy, None, 100, dummy, 65, ctypes.byref(s), dummy, dummy, None, None,
                                      None, 0) == lib.ECHO_ECAPACITY
    s.C = 65536
    assert L.echo_topk_select_cached(1, dummy, None, 100, dummy, 16, None, None, 0.5, dummy, dummy, None, -1,
                                     ctypes.byref(s), dummy, dummy, None, None) == lib.ECHO_EUNSUPPORTED
    s.C = 64
    assert L.echo_topk_select_cached(1, dummy, None, 100, dummy, 16, None, None, 0.5, dummy, dummy, None, -1,
                                     ctypes.byref(s), None, dummy, None, None) == lib.ECHO_EINVAL   # no sel_slot



def test_append_argument_checks(L):
    """echo_append_tokens(B, tok_off, tok_end, n_tokens, k_new, kv_new, k8, ks, cache, status, stream):
    argument errors return before anything is enqueued (no GPU needed)."""
    from sparse_attention_kv_echo_gb300 import lib
    d = ctypes.c_void_p(0x1000)
    assert L.echo_append_tokens(0, d, d, 10, d, d, d, d, None, d, None) == lib.ECHO_EINVAL
    assert L.echo_append_tokens(1, d, d, 0, d, d, d, d, None, d, None) == lib.ECHO_EINVAL
    assert L.echo_append_tokens(1, None, d, 10, d, d, d, d, None, d, None) == lib.ECHO_EINVAL
    assert L.echo_append_tokens(1, d, None, 10, d, d, d, d, None, d, None) == lib.ECHO_EINVAL
    assert L.echo_append_tokens(1, d, d, 10, d, d, d, d, None, d, None) == lib.ECHO_EINVAL   # no cache
    assert L.echo_append_tokens(lib.MAX_REQUESTS + 1, d, d, 10, d, d, d, d, None, d, None) == lib.ECHO_EUNSUPPORTED


def test_pool_argument_checks(L):
    """echo_pool_above / echo_pool_select / echo_pool_slots refuse bad arguments before any launch."""
    from sparse_attention_kv_echo_gb300 import lib
    d = ctypes.c_void_p(0x1000)
    assert L.echo_pool_above(0, d, None, 10, d, None, d, d, None) == lib.ECHO_EINVAL
    assert L.echo_pool_above(1, d, None, 10, d, None, d, d, None) == lib.ECHO_EINVAL      # no pool
    assert L.echo_pool_select(1, None, d, 8, d, None) == lib.ECHO_EINVAL
    assert L.echo_pool_select(1, d, d, 0, d, None) == lib.ECHO_EINVAL
    assert L.echo_pool_slots(lib.MAX_REQUESTS + 1, d, 8, d, d, None) == lib.ECHO_EUNSUPPORTED
    assert L.echo_seed_early(1, d, None, 10, None, 8, d, None, d, None) == lib.ECHO_EINVAL


def test_pool_layer_refuses_append():
    import torch
    from sparse_attention_kv_echo_gb300 import DecodeLayer
    lay = DecodeLayer.__new__(DecodeLayer)
    lay.tok_end, lay.pool_slots = torch.zeros(1, dtype=torch.int64), 64
    with pytest.raises(ValueError):
        lay.append(torch.zeros((1, 128)), torch.zeros((1, 576)))


def test_paged_calls_check_their_arguments(L):
    """echo_mla_chunk, echo_mla_mass, echo_evict_select and echo_cache_release refuse before any CUDA call."""
    from sparse_attention_kv_echo_gb300 import lib
    v = ctypes.c_void_p
    d = v(0x1000)

    def pages(**kw):
        p = lib.EchoPagesStruct()
        p.page_tab, p.kv, p.kv_rows, p.req_rows, p.page = 0x1000, 0x1000, 64, 0, 16
        for k, x in kw.items():
            setattr(p, k, x)
        return ctypes.byref(p)

    def chunk(B=1, row_off=d, n_rows=2, heads=16, q=d, tok_off=d, n=10, pg=None, sel=None, k=0, window=0, sinks=0,
              scale=0.1, out=d, lse=d, ws=d, short=0, status=d):
        size = lib.mla_chunk_workspace_size(max(n_rows, 1), max(heads, 1), max(B, 1))
        return L.echo_mla_chunk(B, row_off, n_rows, heads, q, tok_off, None, n, pages() if pg is None else pg, sel, k,
                                window, sinks, scale, out, lse, ws, size - short, status, None)
    inf, nan = float("inf"), float("nan")
    for bad in (dict(B=0), dict(row_off=None), dict(n_rows=-1), dict(heads=0), dict(q=None), dict(tok_off=None),
                dict(n=-1), dict(window=-1), dict(sinks=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=inf),
                dict(scale=nan), dict(out=None), dict(lse=None), dict(ws=None), dict(short=1), dict(status=None),
                dict(q=v(0x1008)), dict(out=v(0x1004)), dict(ws=v(0x1010)), dict(pg=pages(page=0)),
                dict(pg=pages(page_tab=None)), dict(pg=pages(kv=None)), dict(pg=pages(kv=0x1008)),
                dict(pg=pages(kv_rows=0)), dict(pg=pages(req_rows=-1)), dict(pg=pages(req_rows=65)),
                dict(B=3, pg=pages(req_rows=22)), dict(sel=d, k=0), dict(sel=d, k=-4), dict(sel=d, k=4, window=3),
                dict(sel=d, k=4, sinks=1)):
        assert chunk(**bad) == lib.ECHO_EINVAL, bad
    for big in (dict(B=lib.MAX_REQUESTS + 1), dict(heads=129), dict(n_rows=(1 << 20) + 1)):
        assert chunk(**big) == lib.ECHO_EUNSUPPORTED, big
    assert chunk(n_rows=0, q=None, out=None, lse=None) == lib.ECHO_OK
    assert lib.mla_chunk_workspace_size(-1, 16, 1) == 0 and lib.mla_chunk_workspace_size(4, 0, 1) == 0

    def mass(lse=d, m=d, out=d, decay=0.5, n=10, scale=0.1, n_rows=2, ws=d, short=0):
        return L.echo_mla_mass(1, d, n_rows, 16, d, lse, d, None, n, pages(), 0, 0, scale, m, out, decay, ws,
                               lib.mla_mass_workspace_size(max(n, 0), 1) - short, d, None)
    for bad in (dict(ws=None), dict(ws=v(0x1080)), dict(short=1), dict(lse=None), dict(m=None), dict(out=None), dict(decay=-0.1), dict(decay=nan), dict(decay=inf),
                dict(n=-1), dict(scale=0.0), dict(n_rows=-1)):
        assert mass(**bad) == lib.ECHO_EINVAL, bad
    assert mass(n=0, m=None, out=None) == lib.ECHO_OK

    def evict(B=1, off=d, n=10, s2t=d, C=64, m=d, keep=1, sinks=0, recent=0, et=d, es=d, ec=d, st=d):
        return L.echo_evict_select(B, off, None, n, s2t, C, m, keep, sinks, recent, et, es, ec, st, None)
    for bad in (dict(B=0), dict(off=None), dict(n=-1), dict(s2t=None), dict(C=0), dict(m=None), dict(keep=-1),
                dict(sinks=-1), dict(recent=-1), dict(et=None), dict(es=None), dict(ec=None), dict(st=None)):
        assert evict(**bad) == lib.ECHO_EINVAL, bad
    assert evict(B=lib.MAX_REQUESTS + 1) == lib.ECHO_EUNSUPPORTED
    assert evict(C=(1 << 19) + 1) == lib.ECHO_EUNSUPPORTED

    c = lib.EchoCacheStruct()
    for f, _ in lib.EchoCacheStruct._fields_:
        if f not in ("row_bytes", "C", "reserved"):
            setattr(c, f, 0x1000)
    c.row_bytes, c.C = 1152, 64
    cache = ctypes.byref(c)

    def release(B=1, off=d, n=10, tok=d, m=4, cache=cache, st=d):
        return L.echo_cache_release(B, off, None, n, tok, m, cache, None, st, None)
    for bad in (dict(B=0), dict(off=None), dict(n=-1), dict(tok=None), dict(m=-1), dict(cache=None), dict(st=None)):
        assert release(**bad) == lib.ECHO_EINVAL, bad
    assert release(B=lib.MAX_REQUESTS + 1) == lib.ECHO_EUNSUPPORTED
    assert release(m=0, tok=None) == lib.ECHO_OK
    c.C = 48
    assert release() == lib.ECHO_ECAPACITY
