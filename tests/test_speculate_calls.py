"""The calls of speculative decoding on the CPU: refusals before any CUDA call, and the plain forms themselves."""
import ctypes
import itertools

import pytest
import torch

from sparse_attention_kv_echo_gb300 import _lib as L
from test_paged_calls import host  # noqa: F401  (fixture: the library and the device replaced by recorders)

from _speculate import Pool, ancestors, mask_words, verify

v = ctypes.c_void_p
d = v(0x1000)


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_kv_echo_gb300 import build
    build.build()
    return L.load()


def test_tree_calls_check_their_arguments(lib):
    def masks(B=1, off=d, n=4, parent=d, words=1, mask=d, depth=None, st=d):
        return lib.echo_tree_masks(B, off, n, parent, words, mask, depth, st, None)
    for bad in (dict(B=0), dict(off=None), dict(n=-1), dict(parent=None), dict(words=0), dict(words=-3), dict(mask=None), dict(st=None)):
        assert masks(**bad) == L.ECHO_EINVAL, bad
    for big in (dict(B=L.MAX_REQUESTS + 1), dict(n=(1 << 20) + 1), dict(words=L.TREE_MAX_WORDS + 1)):
        assert masks(**big) == L.ECHO_EUNSUPPORTED, big
    assert masks(n=0, parent=None, mask=None) == L.ECHO_OK

    def pages(**kw):
        p = L.EchoPagesStruct()
        p.page_tab, p.kv, p.kv_rows, p.req_rows, p.page = 0x1000, 0x1000, 64, 0, 16
        for k, x in kw.items():
            setattr(p, k, x)
        return ctypes.byref(p)

    def tree(B=1, row_off=d, n_rows=2, heads=16, q=d, mask=d, words=1, tok_off=d, n=10, pg=None, scale=0.1, out=d, lse=d, ws=d,
             short=0, st=d):
        size = L.mla_chunk_workspace_size(max(n_rows, 1), max(heads, 1), max(B, 1))
        return lib.echo_mla_tree(B, row_off, n_rows, heads, q, mask, words, tok_off, None, n, pages() if pg is None else pg, scale,
                                 out, lse, ws, size - short, st, None)
    for bad in (dict(B=0), dict(row_off=None), dict(n_rows=-1), dict(heads=0), dict(q=None), dict(mask=None), dict(words=0),
                dict(tok_off=None), dict(n=-1), dict(scale=0.0), dict(scale=float("nan")), dict(out=None), dict(lse=None), dict(ws=None),
                dict(short=1), dict(st=None), dict(q=v(0x1008)), dict(out=v(0x1004)), dict(ws=v(0x1010)), dict(pg=pages(page=0)),
                dict(pg=pages(kv=None)), dict(pg=pages(kv_rows=0)), dict(pg=pages(page_tab=None))):
        assert tree(**bad) == L.ECHO_EINVAL, bad
    for big in (dict(B=L.MAX_REQUESTS + 1), dict(heads=129), dict(n_rows=(1 << 20) + 1), dict(words=33)):
        assert tree(**big) == L.ECHO_EUNSUPPORTED, big
    assert tree(n_rows=0, q=None, mask=None, out=None, lse=None) == L.ECHO_OK


def test_verification_checks_its_arguments(lib):
    def call(B=1, off=d, n=4, parent=d, token=d, vocab=100, dtype=0, target=d, draft=d, un=d, up=d, path=d, count=d, nxt=d, st=d):
        return lib.echo_draft_verify(B, off, n, parent, token, vocab, dtype, target, draft, un, up, path, count, nxt, st, None)
    for bad in (dict(B=0), dict(off=None), dict(n=-1), dict(parent=None), dict(token=None), dict(vocab=0), dict(target=None), dict(un=None),
                dict(up=None), dict(path=None), dict(count=None), dict(nxt=None), dict(st=None), dict(target=v(0x1008)), dict(draft=v(0x1004))):
        assert call(**bad) == L.ECHO_EINVAL, bad
    for big in (dict(B=L.MAX_REQUESTS + 1), dict(n=(1 << 20) + 1), dict(vocab=L.MAX_VOCAB + 1), dict(dtype=2), dict(dtype=-1)):
        assert call(**big) == L.ECHO_EUNSUPPORTED, big


def test_page_calls_check_their_arguments(lib):
    def pool(**kw):
        p = L.EchoPagePoolStruct()
        p.page_tab = p.refs = p.kv = 0x1000
        p.n_pages, p.row_bytes, p.layer_bytes, p.layers, p.page = 10, 1152, 10 * 16 * 1152, 2, 16
        for k, x in kw.items():
            setattr(p, k, x)
        return ctypes.byref(p)

    def size(B):
        return L.pages_workspace_size(max(1, min(B, L.MAX_REQUESTS)), 10)
    calls = {
        "reserve": lambda B=1, off=d, end=d, want=d, n=64, p=None, ws=d, short=0, st=d: lib.echo_pages_reserve(
            B, off, end, want, n, p or pool(), None, ws, size(B) - short, st, None),
        "free": lambda B=1, off=d, end=d, n=64, p=None, st=d: lib.echo_pages_free(B, off, end, n, p or pool(), st, None),
        "fork": lambda m=2, src=d, dst=d, B=1, off=d, end=d, n=64, p=None, ws=d, short=0, st=d: lib.echo_pages_fork(
            m, src, dst, B, off, end, n, p or pool(), ws, size(m) - short, st, None),
        "compact": lambda n=64, p=None, used=d, ws=d, short=0, st=d: lib.echo_pages_compact(n, p or pool(), used, ws, size(1) - short, st, None),
        "keep": lambda B=1, ro=d, rows=4, path=d, count=d, off=d, end=d, n=64, p=None, new=v(0x9000), st=d: lib.echo_rows_keep(
            B, ro, rows, path, count, off, end, n, p or pool(), new, st, None)}
    bad_pools = [dict(refs=None), dict(kv=None), dict(page_tab=None), dict(kv=0x1008), dict(n_pages=0), dict(page=0), dict(page=-1), dict(layers=0),
                 dict(row_bytes=8), dict(row_bytes=1160), dict(layer_bytes=10 * 16 * 1152 - 16), dict(layer_bytes=10 * 16 * 1152 + 8),
                 dict(row_bytes=1 << 60)]
    for name, call in calls.items():
        for bad in bad_pools:
            assert call(p=pool(**bad)) == L.ECHO_EINVAL, (name, bad)
        assert call(p=pool(n_pages=(1 << 24) + 1, layer_bytes=1 << 50)) == L.ECHO_EUNSUPPORTED, name
        assert call(n=-1) == L.ECHO_EINVAL and call(st=None) == L.ECHO_EINVAL, name
        if name != "compact":
            for bad in (dict(B=0), dict(off=None), dict(end=None)):
                assert call(**bad) == L.ECHO_EINVAL, (name, bad)
            assert call(B=L.MAX_REQUESTS + 1) == L.ECHO_EUNSUPPORTED, name
        if name in ("reserve", "fork", "compact"):
            for bad in (dict(ws=None), dict(ws=v(0x1010)), dict(short=1)):
                assert call(**bad) == L.ECHO_EINVAL, (name, bad)
    assert calls["reserve"](want=None) == L.ECHO_EINVAL and calls["compact"](used=None) == L.ECHO_EINVAL
    for bad in (dict(m=-1), dict(src=None), dict(dst=None)):
        assert calls["fork"](**bad) == L.ECHO_EINVAL, bad
    assert calls["fork"](m=L.MAX_REQUESTS + 1) == L.ECHO_EUNSUPPORTED and calls["fork"](m=0, src=None, dst=None, ws=None) == L.ECHO_OK
    for bad in (dict(ro=None), dict(rows=-1), dict(path=None), dict(count=None), dict(new=None), dict(new=d), dict(B=4, new=v(0x1018)),
                dict(B=4, new=v(0x0FE8))):                             # (the ends' arrays overlap)
        assert calls["keep"](**bad) == L.ECHO_EINVAL, bad
    assert calls["keep"](rows=(1 << 20) + 1) == L.ECHO_EUNSUPPORTED
    assert L.pages_workspace_size(0, 5) == L.pages_workspace_size(1, 0) == L.pages_workspace_size(4097, 5) == 0
    assert L.pages_workspace_size(1, (1 << 24) + 1) == 0


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_wrappers_refuse_other_types_shapes_and_layouts(host):  # noqa: F811
    off, st = torch.tensor([0, 4]), _i32(1)
    L.tree_masks(off, _i32(4), _i32(4, 2), st, depth=_i32(4))
    for parent, mask, depth in ((_i32(4).long(), _i32(4, 2), None), (_i32(4), _i32(3, 2), None), (_i32(4), _i32(2, 4).T, None),
                                (_i32(4), _i32(4, 2), _i32(5))):
        with pytest.raises(ValueError):
            L.tree_masks(off, parent, mask, st, depth=depth)
    f = torch.zeros(4, 10)
    u, pick = torch.zeros(4), torch.zeros(1)
    ok = dict(draft=f, u_node=u, u_pick=pick)
    L.draft_verify(off, _i32(4), _i32(4), f, _i32(4), _i32(1), _i32(1), st, **ok)
    L.draft_verify(off, _i32(4), _i32(4), f.bfloat16(), _i32(4), _i32(1), _i32(1), st)
    assert [c[1][6] for c in host.calls if c[0] == "echo_draft_verify"] == [L.DTYPE_F32, L.DTYPE_BF16]
    for bad in (dict(draft=f.bfloat16()), dict(u_node=None), dict(u_pick=None), dict(u_node=u.double()), dict(u_pick=torch.zeros(2)),
                dict(draft=torch.zeros(10, 4).T)):
        with pytest.raises(ValueError):
            L.draft_verify(off, _i32(4), _i32(4), f, _i32(4), _i32(1), _i32(1), st, **{**ok, **bad})
    with pytest.raises(ValueError):
        L.draft_verify(off, _i32(4), _i32(4), f.half(), _i32(4), _i32(1), _i32(1), st)
    kv = torch.zeros((2, 5 * 4, 576), dtype=torch.bfloat16)
    for bad in (dict(page=0), dict(page=2 ** 31), dict(page=8), dict(kv=kv[:, :16]), dict(kv=kv.float()), dict(refs=_i32(5).long())):
        with pytest.raises(ValueError):
            L.PagePool(**{**dict(page_tab=_i32(6), refs=_i32(5), kv=kv, page=4), **bad})
    pool = L.PagePool(_i32(6), _i32(5), kv, 4)
    assert (pool.struct.layers, pool.struct.layer_bytes, pool.struct.n_pages) == (2, 20 * 1152, 5)
    assert pool.of_layer(1).kv.data_ptr() == kv[1].data_ptr() and L.PagePool(_i32(6), _i32(5), kv[0], 4).struct.layers == 1
    tok_off, end, ws = torch.tensor([0, 8, 24]), torch.zeros(2, dtype=torch.int64), torch.zeros(4096, dtype=torch.uint8)
    L.pages_free(tok_off, end, 24, pool, st)
    L.pages_reserve(tok_off, end, end, 24, pool, None, ws, st)
    L.pages_fork(_i32(3), _i32(3), tok_off, end, 24, pool, ws, st)
    L.pages_compact(24, pool, _i32(1), ws, st)
    L.rows_keep(torch.zeros(3, dtype=torch.int64), _i32(7), _i32(2), tok_off, end, 24, pool, end.clone(), st)
    calls = (lambda **k: L.pages_free(k.get("off", tok_off), k.get("end", end), k.get("n", 24), pool, k.get("st", st)),
             lambda **k: L.pages_reserve(k.get("off", tok_off), k.get("end", end), end, k.get("n", 24), pool, None, ws, k.get("st", st)),
             lambda **k: L.pages_fork(_i32(3), _i32(3), k.get("off", tok_off), k.get("end", end), k.get("n", 24), pool, ws, k.get("st", st)),
             lambda **k: L.rows_keep(torch.zeros(3, dtype=torch.int64), _i32(7), _i32(2), k.get("off", tok_off), k.get("end", end),
                                     k.get("n", 24), pool, end.clone(), k.get("st", st)))
    for call in calls:
        for bad in (dict(n=25), dict(off=tok_off.int()), dict(end=end[:1]), dict(end=end.int()), dict(st=_i32(2))):
            with pytest.raises(ValueError):
                call(**bad)
    with pytest.raises(ValueError):
        L.pages_compact(25, pool, _i32(1), ws, st)
    with pytest.raises(ValueError):
        L.pages_fork(_i32(3), _i32(2), tok_off, end, 24, pool, ws, st)


# ---------------------------------------------------------------- the plain forms
def test_the_plain_masks():
    assert ancestors([-1, 0, 0, 1, 9, 4]) == [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {4}, {4, 5}]
    m = mask_words([{0, 31}, {32, 63, 64}], 3)
    assert m.tolist() == [[1 - 2 ** 31, 0, 0], [0, 1 - 2 ** 31, 1]]


@pytest.mark.parametrize("parent", [[-1, 0], [-1, 0, 0], [-1, 0, 0, 0], [-1, 0, 1]])
@pytest.mark.parametrize("certain", [False, True])
def test_the_plain_verification_keeps_the_distribution(parent, certain):
    """The distribution of the first token, exactly: over the drafted tokens (with their probabilities) and, in place of
    the uniform numbers, over the intervals that the accept tests cut [0, 1) into."""
    p = torch.tensor([0.5, 0.125, 0.25, 0.125], dtype=torch.float64)
    q = torch.tensor([0.125, 0.25, 0.5, 0.125], dtype=torch.float64)
    V, n = 4, len(parent)
    kids = [i for i in range(1, n) if parent[i] == 0]
    target, draft = p.repeat(n, 1), None if certain else q.repeat(n, 1)
    got = torch.zeros(V, dtype=torch.float64)
    grid = 16                                                          # p and q are multiples of an eighth
    drafted = [(0,) * len(kids)] if certain else list(itertools.product(range(V), repeat=len(kids)))
    for tokens in drafted:
        weight = 1.0 if certain else float(torch.stack([q[x] for x in tokens]).prod())
        token = [0] * n
        for i, x in zip(kids, tokens):
            token[i] = x
        # the first test's border is a multiple of 1/32 here; the later ones' are averaged over a fine grid
        for us in itertools.product([(k + 0.5) / grid for k in range(grid)], repeat=min(len(kids), 2)):
            u = [0.5] * n
            for i, x in zip(kids, us):
                u[i] = x
            for k in range(grid):
                path, behind = verify(parent, token, target, draft, u, (k + 0.5) / grid)
                first = token[path[1]] if len(path) > 1 else behind
                got[first] += weight / grid ** (len(us) + 1)
    assert torch.allclose(got, p, atol=1.0 / grid if len(kids) > 1 else 1e-12)


def test_the_plain_pages():
    kv = torch.arange(2 * 6 * 4, dtype=torch.float64).view(2, 24, 1)
    P = Pool(6, 6, 4, kv.clone())
    off = [0, 12, 24]
    assert P.reserve(off, [0, 12], [5, 13], 24) == [5, 13] and P.tab == [0, 1, -1, 2, -1, -1] and P.refs == [1, 1, 1, 0, 0, 0]
    end = [5, 12]
    P.fork([0], [1], off, end, 24)
    assert end == [5, 17] and P.tab == [0, 1, -1, 0, 2, -1] and P.refs == [2, 1, 1, 0, 0, 0]
    assert torch.equal(P.kv[:, 8], kv[:, 4]) and torch.equal(P.kv[:, 9], kv[:, 9])
    P.free(off, [2, 17], 24)
    assert P.tab == [0, -1, -1, 0, 2, -1] and P.refs == [2, 0, 1, 0, 0, 0]
    assert P.reserve(off, [2, 17], [3, 17], 24) == [3, 17]            # the shared page is copied
    assert P.tab == [1, -1, -1, 0, 2, -1] and P.refs == [1, 1, 1, 0, 0, 0]
    P.free(off, [3, 12], 24)
    assert P.compact() == 1 and P.tab == [0, -1, -1, -1, -1, -1] and P.refs == [1, 0, 0, 0, 0, 0]
    assert P.keep([0, 3, 3], [1, -1, -1], [1, 0], off, [3, 12], 24) == [1, 12] and not P.bad and not P.full
