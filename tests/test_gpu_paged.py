"""Attention of a chunk over a paged latent cache, accumulated attention weights, victims and release
against plain 64-bit forms: ragged batches, head counts, page sizes, windows, selections, absent tokens,
rows that see nothing, streams and graphs."""
import math

import pytest
import torch

import _paged as P
from sparse_attention_kv_echo_gb300 import _lib as L

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    L.load(build_if_missing=True)


def _buffers(n, heads, B):
    out = torch.full((n, heads, L.MLA_DV), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((n, heads), 7.0, dtype=torch.float32, device=dev)
    ws = torch.full((L.mla_chunk_workspace_size(n, heads, B),), 0xFF, dtype=torch.uint8, device=dev)
    return out, lse, ws, torch.zeros(1, dtype=torch.int32, device=dev)


def _attend(bt, window=0, sinks=0, sel=None, status=0):
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    out, lse, ws, st = _buffers(bt.n, bt.heads, len(bt.lens))
    L.mla_chunk(row_off, q, tok_off, bt.n_tokens, pages, bt.scale, out, lse, ws, st, tok_end=tok_end, window=window,
                sinks=sinks, sel=None if sel is None else sel.to(dev))
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return out.cpu(), lse.cpu()


def _compare(bt, got, window=0, sinks=0, sel=None):
    out, lse = got
    ref, rlse, absv, dots = bt.attend(window, sinks, sel)
    fin = torch.isfinite(rlse)
    assert torch.equal(fin, torch.isfinite(lse)), "rows that see nothing"
    assert torch.all(lse[~fin] == -math.inf) and torch.all(out[~fin] == 0)
    n = max(bt.lens + [0 if sel is None else sel.shape[1]])
    e = (lse.double() - rlse).abs()[fin]
    assert torch.all(e <= P.lse_tolerance(dots, rlse, n)[fin]), float(e.max())
    d = (out.double() - ref).abs()
    tol = P.out_tolerance(ref, absv, dots, n)
    assert torch.all(d <= tol), (float((d - tol).max()), torch.nonzero(d > tol)[:4])


CASES = [
    # lens, rows, heads, page
    ([1], [1], 128, 64),                       # a context of one token
    ([5], [5], 128, 1),                        # a prompt's first chunk
    ([63, 64, 65], [1, 1, 1], 128, 64),        # around a tile and a page
    ([200], [3], 128, 48),                     # pages that end inside a tile
    ([1000, 3, 129], [1, 2, 64], 128, 16),     # ragged contexts and chunks
    ([700], [130], 64, 64),                    # two rows to 128 heads
    ([300, 33], [17, 33], 16, 16),             # eight rows together, a ragged last group
    ([260], [50], 24, 7),                      # a head count that does not divide 128, odd pages
    ([150], [140], 1, 3),                      # one head
    ([90, 40], [2, 9], 127, 256),
    ([4500], [1], 128, 64),                    # one request over many splits
    ([2100, 1, 0, 900], [1, 1, 0, 1], 128, 64),
    ([1 + 7 * i % 90 for i in range(40)], [i % 2 for i in range(40)], 128, 16),          # more requests than a warp has lanes
    ([3 + i % 5 for i in range(1100)], [(0, 1, 3)[i % 3] for i in range(1100)], 16, 4),  # more than a block has threads
]


@pytest.mark.parametrize("lens,rows,heads,page", CASES)
def test_causal(lens, rows, heads, page):
    bt = P.Batch(lens, rows, heads, page, seed=len(lens) + heads, lead=5)
    _compare(bt, _attend(bt))


@pytest.mark.parametrize("lens,rows,heads,window,sinks", [
    ([500], [1], 128, 100, 0), ([500], [1], 128, 100, 4), ([500, 90], [3, 90], 128, 64, 70),
    ([700], [200], 16, 33, 5), ([300], [300], 24, 1, 0), ([300], [300], 40, 1, 1), ([400], [70], 64, 1000, 2),
    ([64, 129], [20, 129], 8, 10, 200), ([3000], [1], 128, 2900, 17),
])
def test_window_and_sinks(lens, rows, heads, window, sinks):
    bt = P.Batch(lens, rows, heads, 16, seed=window)
    _compare(bt, _attend(bt, window, sinks), window, sinks)


@pytest.mark.parametrize("heads,page,absent", [(128, 1, 0.4), (16, 1, 0.9), (40, 16, 0.5)])
def test_absent_tokens(heads, page, absent):
    bt = P.Batch([300, 40, 2, 1, 1], [3, 40, 2, 1, 1], heads, page, seed=9, absent=absent)
    bt.tab[bt.tok_off[3] // page] = -1         # a row whose only token is absent
    _compare(bt, _attend(bt))


def test_rows_that_see_nothing_and_rows_outside():
    # request 1 has no tokens but a row, request 2 an empty chunk; two rows of q belong to no request
    bt = P.Batch([40, 2, 30], [1, 2, 0], 128, 16, seed=4)
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    tok_end[1] = tok_off[1]
    q = torch.cat([q, q[:2]])
    out, lse, ws, st = _buffers(bt.n + 2, 128, 3)
    L.mla_chunk(row_off, q, tok_off, bt.n_tokens, pages, bt.scale, out, lse, ws, st, tok_end=tok_end)
    assert int(st.item()) == L.ST_BADDATA      # more rows than tokens
    assert torch.all(out[1:3] == 0) and torch.all(lse[1:3] == -math.inf)
    assert torch.all(out[3:] == 7) and torch.all(lse[3:] == 7)
    ref, rlse, absv, dots = bt.attend()
    assert torch.all((out[:1].cpu().double() - ref[:1]).abs() <= P.out_tolerance(ref, absv, dots, 40)[:1])


@pytest.mark.parametrize("heads", [128, 32])
def test_selections(heads):
    g = torch.Generator().manual_seed(3)
    bt = P.Batch([500, 90], [6, 3], heads, 1, seed=2, absent=0.1)
    k = 97
    sel = torch.full((bt.n, k), -1, dtype=torch.int32)
    for r in range(bt.n):
        b = 0 if r < 6 else 1
        m = [k, 1, 0, 64, 65, 33, k, 0, 5][r]
        sel[r, torch.randperm(k, generator=g)[:m]] = torch.randint(0, bt.lens[b], (m,), generator=g, dtype=torch.int32)
    _compare(bt, _attend(bt, sel=sel), sel=sel)


def test_selection_past_the_end_is_left_out():
    bt = P.Batch([50], [2], 128, 16, seed=2)
    sel = torch.tensor([[0, 3, 50, 7], [2147483647, 1, -5, 1]], dtype=torch.int32)
    _compare(bt, _attend(bt, sel=sel, status=L.ST_BADDATA), sel=sel)


def test_page_outside_the_pool_is_absent():
    bt = P.Batch([200], [2], 128, 16, seed=6)
    good = _attend(bt)
    _compare(bt, good)
    bt.tab[4] = 2 ** 31 - 1
    got = _attend(bt, status=L.ST_BADDATA)
    bt.tab[4] = -1
    _compare(bt, got)


def test_each_request_its_own_rows():
    bt = P.Batch([300, 120, 77], [1, 40, 1], 128, 1, seed=5, per_request=320)
    _compare(bt, _attend(bt))


def test_unseen_rows_may_hold_anything():
    # rows of no token, behind the requests' ends, of absent pages, and out of the window
    bt = P.Batch([300, 50], [1, 1], 128, 1, seed=8)
    seen = torch.zeros(bt.kv.shape[0], dtype=torch.bool)
    for b in range(2):
        seen[bt.cache_row(b, bt.visible(b, 0, 60, 3))] = True
    clean = _attend(bt, 60, 3)
    bt.kv[~seen] = math.nan
    bt.kv[torch.nonzero(~seen)[::2, 0]] = math.inf
    dirty = _attend(bt, 60, 3)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


def test_a_nan_query_stays_in_its_row():
    # the rows packed with it, and the pieces of its own context that are joined, keep to theirs
    for lens, heads in ([300], 16), ([3000], 128):
        bt = P.Batch(lens, [6], heads, 16, seed=3)
        clean = _attend(bt)
        bt.q[2, 5, 7] = math.nan
        bt.q[4, 1, 100] = math.inf
        out, lse = _attend(bt)
        hurt = torch.zeros((6, heads), dtype=torch.bool)
        hurt[2, 5] = hurt[4, 1] = True
        assert torch.all(torch.isnan(out[hurt])) and torch.all(torch.isnan(lse[hurt]))
        assert torch.equal(out[~hurt], clean[0][~hurt]) and torch.equal(lse[~hurt], clean[1][~hurt])


def test_rows_past_4_gib():
    bt = P.Batch([150, 70], [1, 30], 128, 16, seed=13)
    want = _attend(bt)
    row_off, q, tok_off, tok_end, _ = bt.on(dev, L)
    far = 4_000_000 // 16                        # the pages lie from 4.6 GB on
    kv = torch.zeros((far * 16 + bt.kv.shape[0], 576), dtype=torch.bfloat16, device=dev)
    kv[far * 16:] = bt.kv.to(dev)
    pages = L.KVPages((bt.tab + far).to(dev), kv, 16)
    out, lse, ws, st = _buffers(bt.n, 128, 2)
    L.mla_chunk(row_off, q, tok_off, bt.n_tokens, pages, bt.scale, out, lse, ws, st, tok_end=tok_end)
    assert int(st.item()) == 0 and torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])


def test_token_rows_past_2_to_the_31():
    # the second request's region starts behind 2^31 token rows; pages of 1024
    gap, page = 2 ** 31 + 5, 1024
    bt = P.Batch([90, 200], [1, 3], 128, 64, seed=14)
    n = gap + 300
    tab = torch.full((n // page + 1,), -1, dtype=torch.int32)
    tab[0], tab[gap // page] = 1, 0
    kv = torch.randn((2 * page, 576), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    bt.tok_off = torch.tensor([0, gap, n])
    bt.tok_end, bt.n_tokens, bt.tab, bt.kv, bt.page = torch.tensor([90, gap + 200]), n, tab, kv, page
    _compare(bt, _attend(bt))
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    lse = bt.attend()[1].float().to(dev)
    mass = torch.zeros(n, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    L.mla_mass(row_off, q, lse, tok_off, n, pages, bt.scale, mass, mass, st, tok_end=tok_end)
    assert int(st.item()) == 0
    assert abs(float(mass[:90].sum()) - 128) < 128 * 1e-4 and abs(float(mass[gap:gap + 200].sum()) - 3 * 128) < 384 * 1e-4
    assert float(mass[90:gap].abs().max()) == 0.0


def test_two_calls_at_once():
    a, b = P.Batch([2000, 300], [1, 100], 128, 64, seed=15), P.Batch([900], [200], 32, 16, seed=16)
    want = [_attend(x) for x in (a, b)]
    streams, held = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for _ in range(4):
        for x, s in zip((a, b), streams):
            row_off, q, tok_off, tok_end, pages = x.on(dev, L)
            bufs = _buffers(x.n, x.heads, len(x.lens))
            torch.cuda.current_stream().synchronize()
            held.append((bufs, row_off, q, tok_off, tok_end, pages))
    for i, (bufs, row_off, q, tok_off, tok_end, pages) in enumerate(held):
        x = (a, b)[i % 2]
        L.mla_chunk(row_off, q, tok_off, x.n_tokens, pages, x.scale, *bufs, tok_end=tok_end, stream=streams[i % 2])
    torch.cuda.synchronize()
    for i, (bufs, *_) in enumerate(held):
        assert int(bufs[3].item()) == 0
        assert torch.equal(bufs[0].cpu(), want[i % 2][0]) and torch.equal(bufs[1].cpu(), want[i % 2][1])


def test_growing_scores_move_the_maximum():
    # every token outweighs those before it: the running maximum moves in every tile, in both directions of the row order
    for flip in (False, True):
        bt = P.Batch([400], [2], 128, 16, seed=1)
        ramp = torch.linspace(0.0, 40.0, 400)
        if flip:
            ramp = ramp.flip(0)
        rows = bt.cache_row(0, torch.arange(400))
        bt.q[:, :, 0] = 8.0
        bt.kv[rows, 0] = ramp.to(torch.bfloat16)
        _compare(bt, _attend(bt))


def test_another_stream_and_a_replayed_graph():
    bt = P.Batch([700, 20], [1, 20], 128, 64, seed=11)
    want = _attend(bt)
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    out, lse, ws, st = _buffers(bt.n, 128, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (row_off, q, tok_off, bt.n_tokens, pages, bt.scale, out, lse, ws, st)
    L.mla_chunk(*args, tok_end=tok_end, stream=s)
    s.synchronize()
    assert torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.mla_chunk(*args, tok_end=tok_end)
    # the captured call reads the lengths when it is replayed: one request grows, the other shrinks
    for lens in ([701, 20], [130, 22], [700, 20]):
        bt.lens = lens
        bt.tok_end = bt.tok_off[:-1] + torch.tensor(lens)
        tok_end.copy_(bt.tok_end)
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        _compare(bt, (out.cpu(), lse.cpu()))
    assert torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])


def test_repeated_calls_give_the_same_bits():
    bt = P.Batch([3000, 1700, 5], [2, 1, 5], 128, 64, seed=12)
    a, b = _attend(bt), _attend(bt)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------- accumulated weights
def _weigh(bt, decay, window=0, sinks=0, in_place=False, status=0):
    ref, rlse, _, _ = bt.attend(window, sinks)
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    g = torch.Generator().manual_seed(77)
    mass = torch.rand(bt.n_tokens, generator=g)
    lse = rlse.float().to(dev)
    md = mass.to(dev)
    out = md if in_place else torch.full((bt.n_tokens,), 5.0, dtype=torch.float32, device=dev)
    before = out.cpu().clone()
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    L.mla_mass(row_off, q, lse, tok_off, bt.n_tokens, pages, bt.scale, md, out, st, decay=decay, tok_end=tok_end,
               window=window, sinks=sinks)
    assert int(st.item()) == status
    want, err = bt.weigh(rlse.float(), mass, before, decay, window, sinks)
    # each weight: its score's error (SCORE of sum |q k|), the exponential's, fp32 sums of rows * heads terms in any order
    terms = max(bt.rows) * bt.heads + 4
    tol = (P.SCORE * 1.01 + P.EXP) * err + want.abs() * (terms * 2.0 ** -24)
    d = (out.cpu().double() - want).abs()
    assert torch.all(d <= tol), (float((d - tol).max()), torch.nonzero(d > tol)[:4])
    return out.cpu()


@pytest.mark.parametrize("lens,rows,heads,page", CASES)
def test_weights(lens, rows, heads, page):
    _weigh(P.Batch(lens, rows, heads, page, seed=len(lens) + heads, lead=5), 0.9)


@pytest.mark.parametrize("lens,rows,heads,window,sinks,decay,absent", [
    ([500, 90], [3, 90], 128, 64, 70, 1.0, 0.0), ([700], [200], 16, 33, 5, 0.5, 0.3), ([300], [300], 24, 1, 0, 0.0, 0.0),
    ([64, 129], [20, 129], 8, 10, 200, 0.25, 0.9), ([1500], [1], 128, 300, 4, 1.0, 0.5),
])
def test_weights_window(lens, rows, heads, window, sinks, decay, absent):
    _weigh(P.Batch(lens, rows, heads, 1, seed=window, absent=absent), decay, window, sinks, in_place=decay == 1.0)


@pytest.mark.parametrize("window", [2 ** 63 - 1, 2 ** 62, 0x7FFFFF00, 701])
def test_a_window_as_wide_as_any_context_hides_nothing(window):
    bt = P.Batch([700, 90], [200, 1], 16, 16, seed=9)
    for sinks in (0, 2 ** 63 - 1):
        _weigh(bt, 0.5, window, sinks)
        _compare(bt, _attend(bt, window, sinks), window, sinks)


def test_weights_without_decay_read_no_old_mass():
    bt = P.Batch([70], [4], 128, 16, seed=1)
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    ref, rlse, _, _ = bt.attend()
    mass = torch.full((bt.n_tokens,), math.nan, device=dev)
    out = torch.zeros_like(mass)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    L.mla_mass(row_off, q, rlse.float().to(dev), tok_off, bt.n_tokens, pages, bt.scale, mass, out, st, decay=0.0,
               tok_end=tok_end)
    got = out.cpu().double()
    assert torch.all(torch.isfinite(got)) and abs(float(got.sum()) - 4 * 128) < 4 * 128 * 1e-4


def test_weights_sum_to_rows_and_heads():
    bt = P.Batch([900, 300], [1, 40], 128, 64, seed=3)
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    out, lse, ws, st = _buffers(bt.n, 128, 2)
    mass = torch.zeros(bt.n_tokens, device=dev)
    L.mla_chunk(row_off, q, tok_off, bt.n_tokens, pages, bt.scale, out, lse, ws, st, tok_end=tok_end)
    L.mla_mass(row_off, q, lse, tok_off, bt.n_tokens, pages, bt.scale, mass, mass, st, tok_end=tok_end)
    lo, hi = int(bt.tok_off[1]), int(bt.tok_end[1])
    assert abs(float(mass[:900].sum()) - 128) < 128 * 1e-4
    assert abs(float(mass[lo:hi].sum()) - 40 * 128) < 40 * 128 * 1e-4
    assert int(st.item()) == 0


# ---------------------------------------------------------------- victims
def _select(s2t, mass, off, end, keep, sinks, recent, status=0):
    B, C = s2t.shape
    et = torch.full((B, C), 9, dtype=torch.int32, device=dev)
    es, ec = torch.full_like(et, 9), torch.full((B,), 9, dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    L.evict_select(off.to(dev), mass.numel(), s2t.to(dev), mass.to(dev), keep, et, es, ec, st, sinks=sinks, recent=recent,
                   tok_end=end.to(dev))
    assert int(st.item()) == status
    et, es, ec = et.cpu(), es.cpu(), ec.cpu()
    for b in range(B):
        length = int(end[b] - off[b])
        t, s = P.victims(s2t[b], mass, int(off[b]), length, keep, sinks, recent)
        assert int(ec[b]) == len(t)
        assert es[b].tolist() == s + [-1] * (C - len(s)) and et[b].tolist() == t + [-1] * (C - len(t))


@pytest.mark.parametrize("B,C,length,keep,sinks,recent", [
    (1, 1, 1, 0, 0, 0), (2, 32, 40, 5, 0, 0), (3, 64, 64, 64, 0, 0), (3, 1000, 1500, 300, 4, 50), (1, 4096, 5000, 4000, 4, 256),
    (2, 5000, 5000, 0, 0, 0), (2, 700, 900, 0, 10, 20), (1, 40000, 41000, 20000, 1, 1), (1, 100000, 300000, 99000, 4, 64),
    (2, 64, 40, 3, 40, 0), (2, 64, 40, 3, 0, 41),
])
@pytest.mark.parametrize("kind", ["spread", "ties", "signs"])
def test_victims(B, C, length, keep, sinks, recent, kind):
    g = torch.Generator().manual_seed(B * C + keep)
    off = torch.arange(B + 1, dtype=torch.int64) * (length + 3)
    s2t = torch.full((B, C), -1, dtype=torch.int32)
    for b in range(B):
        m = min(C, length) if b == 0 else max(1, min(C, length) * 2 // 3)
        s2t[b, torch.randperm(C, generator=g)[:m]] = torch.randperm(length, generator=g)[:m].to(torch.int32)
    n = B * (length + 3)
    mass = torch.rand(n, generator=g)
    if kind == "ties":
        mass = (mass * 3).floor()
    if kind == "signs":
        mass = (mass * 9).floor() - 4.0
        mass[::3] *= -0.0
        mass[5::97] = math.inf
        mass[7::89] = -math.inf
    _select(s2t, mass, off, off[:-1] + length, keep, sinks, recent)


def test_victims_with_tokens_past_the_end():
    s2t = torch.tensor([[0, 5, 9, 10, -1, 2]], dtype=torch.int32)
    _select(s2t, torch.arange(12.0), torch.tensor([0, 12]), torch.tensor([10]), 1, 0, 0, status=L.ST_BADDATA)


def test_nan_mass_is_reported_and_heaviest():
    s2t = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32)
    mass = torch.tensor([1.0, math.nan, math.inf, 0.0])
    et = torch.empty((1, 4), dtype=torch.int32, device=dev)
    es, ec = torch.empty_like(et), torch.empty(1, dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    L.evict_select(torch.tensor([0, 4], device=dev), 4, s2t.to(dev), mass.to(dev), 1, et, es, ec, st)
    assert int(st.item()) == L.ST_NAN and et.tolist() == [[0, 2, 3, -1]] and int(ec) == 3


# ---------------------------------------------------------------- together, on the library's cache
def test_a_cache_that_shrinks_and_grows():
    """Append, attend, weigh, evict, release on one LayerCache: the tables stay consistent and every result
    is that of the plain forms over the tokens the cache holds."""
    B, C, room, heads = 2, 64, 200, 128
    g = torch.Generator().manual_seed(21)
    off = torch.tensor([0, room, 2 * room], dtype=torch.int64)
    host = torch.zeros((2 * room, 576), dtype=torch.bfloat16).pin_memory()
    cache = L.LayerCache(B, 2 * room, C, host)
    tok_off, tok_end = off.to(dev), off[:-1].clone().to(dev)
    k8 = torch.zeros((2 * room, 128), dtype=torch.uint8, device=dev)
    ks = torch.zeros(2 * room, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    mass = torch.zeros(2 * room, device=dev)
    pages = L.KVPages.of_cache(cache)
    row_off = torch.arange(B + 1, dtype=torch.int64)
    out, lse, ws, _ = _buffers(B, heads, B)
    et = torch.empty((B, C), dtype=torch.int32, device=dev)
    es, ec = torch.empty_like(et), torch.empty(B, dtype=torch.int32, device=dev)
    scale = 1.0 / math.sqrt(192.0)
    ref_mass = torch.zeros(2 * room, dtype=torch.float64)
    for step in range(90):
        kv_new = torch.randn((B, 576), generator=g).to(torch.bfloat16)
        L.append_tokens(tok_off, tok_end, 2 * room, torch.randn((B, 128), generator=g).to(dev), kv_new.to(dev), k8, ks,
                        cache, st)
        q = torch.randn((B, heads, 576), generator=g).to(torch.bfloat16)
        L.mla_chunk(row_off.to(dev), q.to(dev), tok_off, 2 * room, pages, scale, out, lse, ws, st, tok_end=tok_end)
        L.mla_mass(row_off.to(dev), q.to(dev), lse, tok_off, 2 * room, pages, scale, mass, mass, st, decay=0.9,
                   tok_end=tok_end)
        torch.cuda.synchronize()
        t2s = cache.tok2slot.cpu()
        if step % 10 == 9 or step == 0:
            bt = P.Batch.__new__(P.Batch)
            bt.lens, bt.rows, bt.heads, bt.page = [step + 1] * B, [1] * B, heads, 1
            bt.tok_off, bt.tok_end, bt.row_off, bt.n = off, off[:-1] + step + 1, row_off, B
            bt.n_tokens, bt.tab, bt.req_rows, bt.kv, bt.q, bt.scale = 2 * room, t2s, C, cache.dev_kv.cpu(), q, scale
            assert torch.equal(bt.kv[bt.cache_row(0, bt.visible(0, 0))], host[bt.visible(0, 0)])
            _compare(bt, (out.cpu(), lse.cpu()))
        L.evict_select(tok_off, 2 * room, cache.slot2tok, mass, 40, et, es, ec, st, sinks=2, recent=8, tok_end=tok_end)
        before, s2t = mass.cpu(), cache.slot2tok.view(B, C).cpu()
        L.cache_release(tok_off, 2 * room, et, cache, st, mass=mass, tok_end=tok_end)
        torch.cuda.synchronize()
        for b in range(B):
            gone, slots = P.victims(s2t[b], before, int(off[b]), step + 1, 40, 2, 8)
            assert int(ec[b]) == len(gone) and et[b, :len(gone)].tolist() == gone
            now = cache.slot2tok.view(B, C)[b].cpu()
            t2s = cache.tok2slot.cpu()
            want = s2t[b].clone()
            want[slots] = -1
            assert torch.equal(now, want)
            assert all(int(t2s[int(off[b]) + t]) == -1 and float(mass[int(off[b]) + t]) == 0 for t in gone)
            free = cache.freebits.view(B, C // 32)[b].cpu().tolist()
            assert all(((free[s // 32] >> (s % 32)) & 1) == int(now[s] < 0) for s in range(C))
            assert int((now >= 0).sum()) <= 40
    assert int(st.item()) == 0


def test_release_of_repeated_and_absent_tokens():
    host = torch.zeros((40, 576), dtype=torch.bfloat16).pin_memory()
    cache = L.LayerCache(1, 40, 32, host)
    off = torch.tensor([0, 40], device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    cache.tok2slot[3], cache.slot2tok[7] = 7, 3
    cache.tok2slot[9], cache.slot2tok[31] = 31, 9
    cache.freebits[0] = -1 ^ (1 << 7) ^ -(1 << 31)
    L.cache_release(off, 40, torch.tensor([[3, 5, 3, -1, 3]], dtype=torch.int32, device=dev), cache, st)
    assert int(st.item()) == 0
    assert int(cache.tok2slot[3]) == -1 and int(cache.slot2tok[7]) == -1 and int(cache.tok2slot[9]) == 31
    assert int(cache.freebits[0]) & 0xFFFFFFFF == 0x7FFFFFFF
    L.cache_release(off, 40, torch.tensor([[40]], dtype=torch.int32, device=dev), cache, st)
    assert int(st.item()) == L.ST_BADDATA


@pytest.mark.parametrize("what", ["dtype", "shape", "pages", "strides", "sel", "ws"])
def test_wrapper_refuses(what):
    bt = P.Batch([40], [2], 16, 16, seed=1)
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    out, lse, ws, st = _buffers(2, 16, 1)
    sel, n = None, bt.n_tokens
    if what == "dtype":
        q = q.half()
    if what == "shape":
        out = out[:1]
    if what == "pages":
        n = bt.n_tokens + 1000
    if what == "strides":
        q = torch.cat([q, q], -1)[:, :, :576]
    if what == "ws":
        ws = ws.cpu()
    if what == "sel":
        sel = torch.zeros((1, 4), dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        L.mla_chunk(row_off, q, tok_off, n, pages, bt.scale, out, lse, ws, st, tok_end=tok_end, sel=sel)


# ---------------------------------------------------------------- in the framework's own paths
def _plain_selected(q, host, off, sel, scale):
    """A Batch over the host rows, one row each: the attention of the rows over their listed tokens."""
    bt = P.Batch.__new__(P.Batch)
    B = len(off) - 1
    bt.lens, bt.heads, bt.page, bt.req_rows = [int(off[b + 1] - off[b]) for b in range(B)], q.shape[1], 1, 0
    bt.tok_off, bt.tok_end = torch.as_tensor(off), torch.as_tensor(off)[1:]
    bt.n_tokens, bt.n, bt.kv, bt.q, bt.scale = int(off[-1]), q.shape[0], host, q, scale
    bt.rows = [q.shape[0]] if B == 1 else [1] * B
    bt.row_off = torch.tensor([0] + bt.rows).cumsum(0)
    bt.tab = torch.arange(int(off[-1]), dtype=torch.int32)
    return bt


@pytest.mark.parametrize("heads", [128, 16])
def test_prefill_blocks_attend_over_their_selections(heads):
    from sparse_attention_kv_echo_gb300 import workloads as wl
    from sparse_attention_kv_echo_gb300.prefill import PrefillRunner
    w = wl.scaled(wl.WORKLOADS["prefill"], "attn", lengths=(700,), k=96, C=704, prefill_block=200)
    k8, ks = wl.make_keys(w, 0)
    host = wl.make_host_pool(w, 0, pin=True)
    pr = PrefillRunner(k8.to(dev), ks.to(dev), w.k, w.C, host, w.prefill_block, attention=True, heads=heads)
    g = torch.Generator().manual_seed(5)
    got = []
    for i in range(pr.blocks()):                     # enqueued back to back: block i attends beside block i + 1
        q, wt = wl.make_prefill_queries(w, i)
        mq = torch.randn((q.shape[0], heads, 576), generator=g).to(torch.bfloat16)
        _, R = pr.block(i, q.to(dev), wt.to(dev), mla_q=mq.to(dev))
        with torch.cuda.stream(pr.copy):
            got.append((mq, pr.sel_idx[:R].clone(), pr.attn_out[:R].clone(), pr.attn_lse[:R].clone()))
    torch.cuda.synchronize()
    assert int(pr.status.item()) == 0
    for i, (mq, sel, out, lse) in enumerate(got):
        rows = torch.tensor([0, 1, len(mq) // 2, len(mq) - 1])
        sel = sel.cpu()
        p = i * w.prefill_block + rows
        assert torch.all((sel[rows] >= 0).sum(1) == torch.clamp(p + 1, max=w.k))
        bt = _plain_selected(mq[rows], host, [0, w.total_tokens], sel[rows], pr.mla_scale)
        _compare(bt, (out.cpu()[rows], lse.cpu()[rows]), sel=sel[rows])
    with pytest.raises(ValueError):
        pr.block(0, q.to(dev), wt.to(dev))


@pytest.mark.parametrize("hold_early,graph", [(False, True), (True, False)])
def test_a_shared_pool_attends(hold_early, graph):
    from sparse_attention_kv_echo_gb300 import DecodeLayer
    from sparse_attention_kv_echo_gb300 import workloads as wl
    w = wl.scaled(wl.WORKLOADS["batch"], "poolattn", B=3, lengths=(1500, 90, 2100), k=128, C=512)
    off = wl.tok_offsets(w.lengths)
    k8, ks = wl.make_keys(w, 0)
    host = wl.make_host_pool(w, 0, pin=True)
    lay = DecodeLayer(off, k8.to(dev), ks.to(dev), w.k, w.C, host, pool_slots=1024, hold_early=hold_early, attention=True)
    main = torch.cuda.Stream()
    lay.w_in.copy_(wl.make_weights(w, 0).to(dev))
    torch.cuda.synchronize()
    if graph:
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg, stream=main):
            lay.step(stream=main)
        torch.cuda.synchronize()
        lay.reset()
    qs = wl.QueryStream(w, 0)
    g = torch.Generator().manual_seed(9)
    for _ in range(3):
        mq = torch.randn((3, L.MLA_HEADS, 576), generator=g).to(torch.bfloat16)
        with torch.cuda.stream(main):
            lay.q_in.copy_(qs.next().to(dev))
            lay.mla_q.copy_(mq.to(dev))
            cg.replay() if graph else lay.step(stream=main)
        torch.cuda.synchronize()
        assert int(lay.status.item()) == 0
        sel = lay.sel_idx.cpu()
        bt = _plain_selected(mq, host, off, sel, lay.mla_scale)
        _compare(bt, (lay.attn_out.cpu(), lay.attn_lse.cpu()), sel=sel)


@pytest.mark.parametrize("B", [3, 32, 33])
def test_a_pool_steps_launches_are_what_it_says(B):
    from torch.profiler import ProfilerActivity, profile
    from sparse_attention_kv_echo_gb300 import DecodeLayer
    from sparse_attention_kv_echo_gb300 import workloads as wl
    w = wl.scaled(wl.WORKLOADS["batch"], "poolcount", B=B, lengths=(300,) * B, k=64, C=128)
    k8, ks = wl.make_keys(w, 0)
    host = wl.make_host_pool(w, 0, pin=True)
    off, q = wl.tok_offsets(w.lengths), wl.QueryStream(w, 0).next().to(dev)
    said, ran = [], []
    with profile(activities=[ProfilerActivity.CUDA]):  # a process's first session may come out empty
        torch.zeros(1, device=dev)
        torch.cuda.synchronize()
    for attention in (False, True):
        lay = DecodeLayer(off, k8.to(dev), ks.to(dev), w.k, w.C, host, pool_slots=B * 96, attention=attention)
        lay.w_in.copy_(wl.make_weights(w, 0).to(dev))
        lay.q_in.copy_(q)
        lay.step()
        torch.cuda.synchronize()
        with profile(activities=[ProfilerActivity.CUDA]) as prof:
            lay.step()
            torch.cuda.synchronize()
        assert int(lay.status.item()) == 0
        said.append(lay.kernel_launches_per_step())
        ran.append(sum("echo::" in e.name and e.device_type == torch.autograd.DeviceType.CUDA for e in prof.events()))
    assert said == ran
    assert said[1] - said[0] == (2 if B <= 32 else 3)
