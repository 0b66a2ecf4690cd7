"""More of the calls over a paged latent cache: workspaces on other streams, caches under lazy reuse, long
pieces of work, rows that add nothing, the sizes that are measured, by samples, and
captured, empty and first calls."""
import numpy as np
import pytest
import torch

import _paged as P
from sparse_attention_kv_echo_gb300 import _lib as L

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    L.load(build_if_missing=True)


def _weigh(bt, lse, mass, stream=None, ws=None):
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    out = torch.zeros_like(mass)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()

    def call():
        L.mla_mass(row_off, q, lse, tok_off, bt.n_tokens, pages, bt.scale, mass, out, st, decay=0.5, tok_end=tok_end,
                   stream=stream, ws=ws)
    return call, out, st


def test_weights_on_another_stream_take_a_workspace_of_that_stream():
    # a block of the workspace's size is freed on the current stream while the kernel that fills it is still pending
    # there: the call on the other stream does not get it
    bt = P.Batch([900, 300], [1, 40], 128, 64, seed=3)
    lse = bt.attend()[1].float().to(dev)
    mass = torch.rand(bt.n_tokens, device=dev)
    size = L.mla_mass_workspace_size(bt.n_tokens, 2)
    call, want, st = _weigh(bt, lse, mass, ws=torch.zeros(size, dtype=torch.uint8, device=dev))
    call()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    call, got, st2 = _weigh(bt, lse, mass, stream=other)
    for cycles in (0, 20_000, 100_000):
        block = torch.empty(size, dtype=torch.uint8, device=dev)
        torch.cuda._sleep(cycles)
        block.zero_()
        del block
        call()
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and int(st2.item()) == 0
        assert torch.equal(got, want)


# ---------------------------------------------------------------- caches under lazy reuse
def _lazy_cache(n=200, C=64, keep=20):
    """One request of n tokens whose cache of C slots holds `keep` residents and, in every other slot, a ghost."""
    host = torch.zeros((n, 576), dtype=torch.bfloat16).pin_memory()
    cache = L.LayerCache(1, n, C, host)
    off = torch.tensor([0, n], device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    slots = torch.empty((1, C), dtype=torch.int32, device=dev)
    first = torch.arange(3, 3 + 2 * C, 2, dtype=torch.int32, device=dev)[None]
    L.cache_step(off, n, first, cache, slots, st, lazy=True)
    left = torch.full_like(first, -1)
    left[0, :keep] = first[0, C - 2 * keep::2]
    L.cache_step(off, n, left, cache, slots, st, lazy=True)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    free = cache.freebits.cpu()
    held = torch.tensor([not (int(free[s // 32]) >> (s % 32)) & 1 for s in range(C)])
    assert int(held.sum()) == keep and torch.all(cache.slot2tok >= 0)
    return cache, off, st, held


@pytest.mark.parametrize("keep,sinks,recent", [(40, 0, 0), (20, 0, 0), (7, 0, 0), (0, 60, 80), (3, 10, 10)])
def test_victims_of_a_lazy_cache_are_residents(keep, sinks, recent):
    cache, off, st, held = _lazy_cache()
    mass = torch.rand(200, generator=torch.Generator().manual_seed(keep)).to(dev)
    s2t = cache.slot2tok.cpu()
    mass[s2t[~held].long().to(dev)] = float("nan")         # a ghost's mass is not looked at
    et = torch.full((1, 64), 9, dtype=torch.int32, device=dev)
    es, ec = torch.full_like(et, 9), torch.full((1,), 9, dtype=torch.int32, device=dev)
    L.evict_select(off, 200, cache.slot2tok, mass, keep, et, es, ec, st, sinks=sinks, recent=recent, freebits=cache.freebits)
    t, s = P.victims(torch.where(held, s2t, -1), mass.cpu(), 0, 200, keep, sinks, recent)
    assert int(st.item()) == 0 and int(ec) == len(t)
    assert et[0].tolist() == t + [-1] * (64 - len(t)) and es[0].tolist() == s + [-1] * (64 - len(s))


@pytest.mark.parametrize("B,C,length", [(2, 5024, 6000), (1, 100000, 120000)])
def test_victims_with_free_bits_of_longer_caches(B, C, length):
    g = torch.Generator().manual_seed(C)
    off = torch.arange(B + 1) * length
    s2t = torch.stack([torch.randperm(length, generator=g)[:C] for _ in range(B)]).to(torch.int32)
    free = torch.rand((B, C), generator=g) < 0.3
    bits = (free.view(B, C // 32, 32).long() << torch.arange(32)).sum(2)
    bits = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32).flatten()
    mass = (torch.rand(B * length, generator=g) * 50).floor()
    et = torch.empty((B, C), dtype=torch.int32, device=dev)
    es, ec, st = torch.empty_like(et), torch.empty(B, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    L.evict_select(off.to(dev), B * length, s2t.to(dev), mass.to(dev), C // 3, et, es, ec, st, sinks=4, recent=9,
                   freebits=bits.to(dev))
    assert int(st.item()) == 0
    for b in range(B):
        t, s = P.victims(torch.where(free[b], -1, s2t[b]), mass, int(off[b]), length, C // 3, 4, 9)
        assert int(ec[b]) == len(t) and es[b].tolist() == s + [-1] * (C - len(s)) and et[b].tolist() == t + [-1] * (C - len(t))


def test_release_leaves_freed_tokens_of_a_lazy_cache():
    cache, off, st, held = _lazy_cache()
    t2s, s2t, free = cache.tok2slot.cpu(), cache.slot2tok.cpu(), cache.freebits.cpu()
    mass = torch.arange(1.0, 201.0, device=dev)
    L.cache_release(off, 200, cache.slot2tok.clone()[None], cache, st, mass=mass)      # every token of the cache
    assert int(st.item()) == 0
    gone = s2t[held].long()
    t2s[gone], s2t[held] = -1, -1
    assert torch.equal(cache.tok2slot.cpu(), t2s) and torch.equal(cache.slot2tok.cpu(), s2t)
    assert torch.all(cache.freebits == -1)
    want = torch.arange(1.0, 201.0)
    want[gone] = 0.0
    assert torch.equal(mass.cpu(), want)


def test_release_reports_tables_that_disagree_and_leaves_them():
    host = torch.zeros((40, 576), dtype=torch.bfloat16).pin_memory()
    cache = L.LayerCache(1, 40, 32, host)
    off = torch.tensor([0, 40], device=dev)
    mass = torch.ones(40, device=dev)
    cache.freebits[0] = 0
    cache.tok2slot[3], cache.slot2tok[7] = 7, 4             # slot 7 says another token
    cache.tok2slot[5] = 32                                  # no such slot
    cache.tok2slot[6], cache.slot2tok[8] = 8, 6
    before = cache.tok2slot.cpu()
    for bad in 3, 5:
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        L.cache_release(off, 40, torch.tensor([[bad, 6 if bad == 5 else -1]], dtype=torch.int32, device=dev), cache, st, mass=mass)
        assert int(st.item()) == L.ST_BADDATA
    before[6] = -1
    assert torch.equal(cache.tok2slot.cpu(), before)
    assert int(cache.slot2tok[7]) == 4 and int(cache.slot2tok[8]) == -1 and int(cache.freebits[0]) == 1 << 8
    assert float(mass.sum()) == 39.0 and float(mass[6]) == 0.0


def test_a_token_listed_many_times_is_released_once_and_is_no_bad_data():
    B, n, C = 3, 500, 64
    host = torch.zeros((B * n, 576), dtype=torch.bfloat16).pin_memory()
    off = torch.arange(B + 1, device=dev) * n
    g = torch.Generator().manual_seed(2)
    for _ in range(8):
        cache = L.LayerCache(B, B * n, C, host)
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        sel = torch.stack([torch.randperm(n, generator=g)[:C].sort().values for _ in range(B)]).to(torch.int32)
        slots = torch.empty((B, C), dtype=torch.int32, device=dev)
        L.cache_step(off, B * n, sel.to(dev), cache, slots, st)
        tok = torch.stack([r[:20].repeat(60)[torch.randperm(1200, generator=g)] for r in sel])
        L.cache_release(off, B * n, tok.to(dev), cache, st)
        assert int(st.item()) == 0
        s2t = cache.slot2tok.cpu().view(B, C)
        for b in range(B):
            assert sorted(s2t[b][s2t[b] >= 0].tolist()) == sel[b, 20:].tolist()
        assert int((cache.tok2slot >= 0).sum()) == B * (C - 20)


def test_append_to_a_lazy_cache_drops_the_token_its_slot_held():
    n, C = 160, 64
    host = torch.randn((n, 576), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).pin_memory()
    cache = L.LayerCache(1, n, C, host)
    off, end = torch.tensor([0, n], device=dev), torch.tensor([150], device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    slots = torch.empty((1, C), dtype=torch.int32, device=dev)
    first = torch.arange(0, C, dtype=torch.int32, device=dev)[None]
    L.cache_step(off, n, first, cache, slots, st, lazy=True, tok_end=end)
    left = torch.full_like(first, -1)
    left[0, :24] = first[0, 40:]
    L.cache_step(off, n, left, cache, slots, st, lazy=True, tok_end=end)
    k8, ks = torch.zeros((n, 128), dtype=torch.uint8, device=dev), torch.zeros(n, device=dev)
    for i in range(5):
        kv = torch.randn((1, 576), device=dev).to(torch.bfloat16)
        L.append_tokens(off, end, n, torch.randn((1, 128), device=dev), kv, k8, ks, cache, st)
        t2s, s2t = cache.tok2slot.cpu(), cache.slot2tok.cpu()
        assert int(t2s[150 + i]) == i and int(t2s[i]) == -1
        held = torch.nonzero(s2t >= 0)[:, 0]
        assert torch.equal(t2s[s2t[held].long()].long(), held)                        # the tables are inverse
        assert torch.equal(cache.dev_kv[held.to(dev)].cpu(), host[s2t[held].long()])    # and say what the rows are
    # the dropped tokens, selected again, are recalled: their slots hold others
    sel = torch.full_like(first, -1)
    sel[0, :10] = torch.cat([torch.arange(5), torch.arange(150, 155)]).to(torch.int32)
    L.cache_step(off, n, sel, cache, slots, st, lazy=True, tok_end=end)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(cache.dev_kv[slots[0, :10].long()].cpu(), host[sel[0, :10].long().cpu()])


def test_a_cache_step_right_behind_a_release_or_an_append_sees_its_tables(orc):
    # nothing between the calls: the step's look at the tables before its wait comes after their writes
    B, n, C, k = 4, 900, 512, 200
    host = torch.zeros((B * n, 576), dtype=torch.bfloat16).pin_memory()
    off = torch.arange(B + 1, device=dev) * n
    cache = L.LayerCache(B, B * n, C, host)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    slots = torch.empty((B, k), dtype=torch.int32, device=dev)
    k8, ks = torch.zeros((B * n, 128), dtype=torch.uint8, device=dev), torch.zeros(B * n, device=dev)
    k_new, kv = torch.ones((B, 128), device=dev), torch.zeros((B, 576), dtype=torch.bfloat16, device=dev)
    end = off[:-1] + 800
    g = torch.Generator().manual_seed(6)
    t2s = [np.full(n, -1, np.int32) for _ in range(B)]
    s2t = [np.full(C, -1, np.int32) for _ in range(B)]
    pick = lambda m: torch.stack([torch.randperm(800, generator=g)[:m].sort().values for _ in range(B)]).to(torch.int32)
    for step in range(60):
        sel, tok = pick(k), pick(400)
        sel_d, tok_d = sel.to(dev), tok.to(dev)
        torch.cuda.synchronize()
        if step % 2:
            L.cache_release(off, B * n, tok_d, cache, st)
        else:
            L.append_tokens(off, end, B * n, k_new, kv, k8, ks, cache, st)
        L.cache_step(off, B * n, sel_d, cache, slots, st)
        for b in range(B):
            if step % 2:
                for t in tok[b].tolist():
                    if t2s[b][t] >= 0:
                        s2t[b][t2s[b][t]] = -1
                        t2s[b][t] = -1
            else:
                s = int(np.argmax(s2t[b] < 0))
                t2s[b][800 + step // 2], s2t[b][s] = s, 800 + step // 2
            want = orc.cache_step(sel[b].numpy(), t2s[b], s2t[b])[0]
            assert np.array_equal(slots[b].cpu().numpy(), want), step
        assert np.array_equal(cache.slot2tok.cpu().numpy(), np.concatenate(s2t))
        assert np.array_equal(cache.tok2slot.cpu().numpy(), np.concatenate(t2s))
    assert int(st.item()) == 0


# ---------------------------------------------------------------- long pieces of work
@pytest.fixture
def short_waits():
    # a step of the kernels takes 1 to 4 us; the pieces of these tests take 600 us and more
    L.debug_wait_limit(200_000)
    yield
    L.debug_wait_limit(-1)


def _shared_pages(n, rows, heads, page, seed):
    """One request of n tokens, all of whose pages are one: a token's cache row is its offset in the page."""
    bt = P.Batch([page], [1], heads, page, seed=seed, room=0)
    g = torch.Generator().manual_seed(seed + 1)
    bt.lens, bt.rows, bt.n = [n], [rows], rows
    bt.q = torch.randn((rows, heads, 576), generator=g).to(torch.bfloat16)
    bt.tok_off, bt.tok_end, bt.row_off = torch.tensor([0, n]), torch.tensor([n]), torch.tensor([0, rows])
    bt.n_tokens, bt.tab = n, torch.zeros(-(-n // page), dtype=torch.int32)
    return bt


def test_a_piece_of_attention_longer_than_the_wait_limit(short_waits):
    # 160 rows of 128 heads: every cluster has whole rows, of 60000 tokens (about 750 us) each
    page, n, rows = 256, 60_000, 160
    bt = _shared_pages(n, rows, 128, page, 3)
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    out = torch.empty((rows, 128, 512), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((rows, 128), device=dev)
    ws = torch.empty(L.mla_chunk_workspace_size(rows, 128, 1), dtype=torch.uint8, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    L.mla_chunk(row_off, q, tok_off, n, pages, bt.scale, out, lse, ws, st, tok_end=tok_end)
    assert int(st.item()) == 0
    kv = bt.kv[:page].double()
    for i in (0, 77, 159):
        p = n - rows + i                                 # sees tokens 0 .. p: each cache row so many times
        times = torch.full((page,), (p + 1) // page, dtype=torch.float64)
        times[:(p + 1) % page] += 1
        s = bt.scale * bt.q[i].double() @ kv.T
        ref = torch.logsumexp(s + times.log(), -1)
        w = torch.exp(s - ref[:, None]) * times
        dots = bt.scale * (bt.q[i].double().abs() @ kv.abs().T).amax(-1)
        assert torch.all((lse[i].cpu().double() - ref).abs() <= P.lse_tolerance(dots, ref, n))
        want, absv = w @ kv[:, :512], w @ kv[:, :512].abs()
        assert torch.all((out[i].cpu().double() - want).abs() <= P.out_tolerance(want, absv, dots, n))


def test_an_item_of_weights_longer_than_the_wait_limit(short_waits):
    # the first tokens, seen by all 32768 rows of 16 heads (2048 blocks of about 3.3 us for each 256 tokens); a window
    # of 1 leaves the other tokens only their own row.  256 first tokens an item, three items a cluster
    rows, heads, page = 32768, 16, 256
    sinks = 3 * 256 * (L.sm_count() // 2)
    n = sinks + rows
    bt = _shared_pages(n, rows, heads, page, 5)
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    lse = torch.full((rows, heads), 8.0, device=dev)
    mass = torch.zeros(n, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    L.mla_mass(row_off, q, lse, tok_off, n, pages, bt.scale, mass, mass, st, tok_end=tok_end, window=1, sinks=sinks)
    assert int(st.item()) == 0
    kv, qd = bt.kv[:page].to(dev).double(), q.double()
    s = bt.scale * qd.view(-1, 576) @ kv.T - 8.0
    want = s.exp_().view(rows, heads, page).sum((0, 1)).cpu()
    # (a score is off by up to 2^-17 of scale * sum |q k|, about 27 +- 1: 2.2e-4 of its weight; the exponential and the
    # sums, 64 terms long and compensated beyond, add 2e-5)
    got = mass[:sinks].cpu().double().view(-1, page)
    assert torch.all((got - want).abs() <= 3e-4 * want)


def _counted(bt, i, window=0, sinks=0, sel=None):
    """Row i's (lse, out, absv, dots) in 64 bits, from how often each cache row is seen."""
    t = bt.visible(0, i, window, sinks, sel)
    times = torch.bincount(bt.cache_row(0, t), minlength=bt.kv.shape[0]).double()
    there = times > 0
    kv, times, q = bt.kv[there].double(), times[there], bt.q[i].double()
    s = bt.scale * q @ kv.T
    lse = torch.logsumexp(s + times.log(), -1)
    w = torch.exp(s - lse[:, None]) * times
    return lse, w @ kv[:, :512], w @ kv[:, :512].abs(), bt.scale * (q.abs() @ kv.abs().T).amax(-1)


def _attend_long(bt, **kw):
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    out = torch.full((bt.n, bt.heads, 512), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((bt.n, bt.heads), 7.0, device=dev)
    ws = torch.full((L.mla_chunk_workspace_size(bt.n, bt.heads, 1),), 0xFF, dtype=torch.uint8, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    L.mla_chunk(row_off, q, tok_off, bt.n_tokens, pages, bt.scale, out, lse, ws, st, tok_end=tok_end, **kw)
    assert int(st.item()) == 0
    return out.cpu(), lse.cpu()


def test_values_of_one_sign_over_a_million_tokens():
    # every accumulation may cut off two of the sum's last bits (2^-22): over the 2048 of a leg, the sum growing
    # evenly, at most 2^-12 on the mean; the roundings of weights and results have no sign
    n, rows = 1 << 20, 160
    bt = _shared_pages(n, rows, 128, 4096, 7)
    bt.kv[:, :512] = bt.kv[:, :512].abs()
    out, lse = _attend_long(bt)
    for i in (0, 80, 159):
        ref, want, absv, dots = _counted(bt, i)
        assert torch.all((lse[i].double() - ref).abs() <= P.SCORE * dots + P.EXP * (1 + ref.abs()))
        off = (out[i].double() - want) / absv
        assert abs(float(off.mean())) <= 2.0 ** -12
        assert torch.all(off.abs() <= 2.0 ** -8 + 2 * P.SCORE * dots[:, None] * 1.01 + 2.0 ** -8 + 2.0 ** -10)


@pytest.mark.parametrize("heads,kind", [(128, "rising"), (128, "falling"), (128, "empty"), (16, "rising"), (40, "window"),
                                        (128, "nan"), (128, "listed")])
def test_pieces_of_several_legs(heads, kind):
    # 40000 to 100000 tokens a row, more rows than clusters: pieces of several legs, whole ones and ones that are joined
    page = 512
    per, kw = 128 // heads, {}
    n, rows = (100_000 if kind != "listed" else 600), 160 * per
    bt = _shared_pages(n, rows, heads, page, 11)
    g = torch.Generator().manual_seed(4)
    pages = -(-n // page)
    bt.kv = torch.randn((4 * page, 576), generator=g).to(torch.bfloat16)
    order = torch.arange(pages) * 4 // pages                  # page 0 first, page 3 last
    bt.tab = (order if kind != "falling" else 3 - order).to(torch.int32)
    for i in range(4):                                        # longer keys, larger maxima
        bt.kv[i * page:(i + 1) * page] *= 0.5 + 0.5 * i
    if kind == "empty":                                       # a row sees nothing in its first and third quarters
        bt.tab[(order == 0) | (order == 2)] = -1
    if kind == "window":
        kw = dict(window=70_000, sinks=50)
    if kind == "nan":
        bt.q[5, 3, 9] = float("nan")
    sel = None
    if kind == "listed":
        sel = torch.randint(0, n, (rows, 40_000), generator=g, dtype=torch.int32)
        sel[torch.rand(sel.shape, generator=g) < 0.1] = -1
        kw = dict(sel=sel.to(dev))
    out, lse = _attend_long(bt, **kw)
    again = _attend_long(bt, **kw)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16))
    assert torch.equal(lse.view(torch.int32), again[1].view(torch.int32))
    for i in sorted({0, 1, 5, rows // 3, rows // 2, rows - 2, rows - 1}):
        ref, want, absv, dots = _counted(bt, i, kw.get("window", 0), kw.get("sinks", 0), sel)
        hurt = torch.isnan(ref)
        assert torch.equal(hurt, torch.isnan(lse[i])) and torch.all(torch.isnan(out[i][hurt]))
        ok = ~hurt
        tol = P.lse_tolerance(dots, ref, 0)
        assert torch.all((lse[i].double() - ref).abs()[ok] <= tol[ok])
        tol = P.out_tolerance(want, absv, dots, 0) + absv * 2.0 ** -11
        assert torch.all((out[i].double() - want).abs()[ok] <= tol[ok]), (i, float(((out[i].double() - want).abs() / tol)[ok].max()))


# ---------------------------------------------------------------- rows that add nothing
@pytest.mark.parametrize("heads,rows", [(128, 5), (16, 200), (40, 33)])
def test_a_row_without_lse_adds_no_weight_whatever_its_query_holds(heads, rows):
    # a padded batch: rows whose lse is -inf, their queries never written
    bt = P.Batch([600, 90], [rows, 1], heads, 16, seed=heads)
    lse = bt.attend()[1].float()
    out = torch.arange(rows + 1) % 3 == 1
    lse[out] = -float("inf")
    g = torch.Generator().manual_seed(1)
    mass = torch.rand(bt.n_tokens, generator=g)
    bt.q[out] = 0.0
    call, clean, st = _weigh(bt, lse.to(dev), mass.to(dev))
    call()
    for junk in float("nan"), float("inf"), -float("inf"):
        bt.q[out] = junk
        call, got, st2 = _weigh(bt, lse.to(dev), mass.to(dev))
        call()
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and int(st2.item()) == 0
        assert torch.equal(got, clean) and torch.all(torch.isfinite(got))


# ---------------------------------------------------------------- at the sizes that are measured
def _samples(bt, out, lse, rows, window=0, sinks=0, sel=None):
    """Compares sampled rows (request, row) with their 64-bit values."""
    for b, i in rows:
        r = int(bt.row_off[b]) + i
        t = bt.visible(b, i, window, sinks, sel)
        k, q = bt.kv[bt.cache_row(b, t)].double(), bt.q[r].double()
        s = bt.scale * q @ k.T
        ref = torch.logsumexp(s, -1)
        w = torch.exp(s - ref[:, None])
        dots = bt.scale * (q.abs() @ k.abs().T).amax(-1)
        assert torch.all((lse[r].double() - ref).abs() <= P.lse_tolerance(dots, ref, t.numel()))
        want, absv = w @ k[:, :512], w @ k[:, :512].abs()
        assert torch.all((out[r].double() - want).abs() <= P.out_tolerance(want, absv, dots, t.numel())), (b, i)


def _run_attention(bt, sel=None, **kw):
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    got = []
    for _ in range(2):
        out = torch.full((bt.n, bt.heads, 512), 7.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full((bt.n, bt.heads), 7.0, device=dev)
        ws = torch.full((L.mla_chunk_workspace_size(bt.n, bt.heads, len(bt.lens)),), 0xFF, dtype=torch.uint8, device=dev)
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        L.mla_chunk(row_off, q, tok_off, bt.n_tokens, pages, bt.scale, out, lse, ws, st, tok_end=tok_end,
                    sel=None if sel is None else sel.to(dev), **kw)
        assert int(st.item()) == 0
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])     # the same bits again
    return got[0][0].cpu(), got[0][1].cpu()


def test_a_block_of_2048_rows_over_8192_tokens():
    bt = P.Batch([8192], [2048], 128, 64, seed=31)
    _samples(bt, *_run_attention(bt), [(0, i) for i in (0, 1, 555, 1024, 2046, 2047)])
    out, lse = _run_attention(bt, window=1024, sinks=16)
    _samples(bt, out, lse, [(0, i) for i in (0, 700, 2047)], 1024, 16)


def test_one_row_of_each_of_32_ragged_requests():
    lens = [int(round(1024 * 16 ** (b / 31))) for b in range(32)]
    bt = P.Batch(lens, [1] * 32, 128, 64, seed=32)
    out, lse = _run_attention(bt)
    _samples(bt, out, lse, [(b, 0) for b in (0, 1, 15, 16, 30, 31)])
    out, lse = _run_attention(bt, window=4096, sinks=4)
    _samples(bt, out, lse, [(b, 0) for b in (0, 16, 31)], 4096, 4)


@pytest.mark.parametrize("heads", [128, 16])
def test_1024_rows_of_2048_listed_tokens(heads):
    bt = P.Batch([32768], [1024], heads, 1, seed=33)
    g = torch.Generator().manual_seed(9)
    sel = torch.randint(0, 32768 - 1024, (1024, 2048), generator=g, dtype=torch.int32)
    out, lse = _run_attention(bt, sel=sel)
    _samples(bt, out, lse, [(0, i) for i in (0, 3, 511, 1023)], sel=sel)


@pytest.mark.parametrize("lens,rows,heads,absent", [([8192], [1024], 128, 0.0), ([2048, 4096, 8192], [1, 1, 1], 128, 0.25),
                                                     ([3000, 700], [40, 1], 16, 0.0), ([1500], [1], 1, 0.0)])
def test_weights_are_within_1e5_of_the_64_bit_ones(lens, rows, heads, absent):
    # the header's bound.  What is in it: scores 5e-7 of their size off (|s| up to 12: 6e-6), the score and -lse in
    # units of log2 rounded to 2^-24 of up to 24 (1.4e-6 each, times log 2), the exponential 2^-22, the sums 4e-6 at
    # 64 terms of one sign in the worst order, their roundings of both signs in fact
    bt = P.Batch(lens, rows, heads, 1 if absent else 64, seed=34, absent=absent)
    out, lse = _run_attention(bt)
    g = torch.Generator().manual_seed(3)
    mass = torch.rand(bt.n_tokens, generator=g)
    call, got, st = _weigh(bt, lse.to(dev), mass.to(dev))
    call()
    assert int(st.item()) == 0
    got = got.cpu().double() - 0.5 * mass.double()
    for b in range(len(lens)):
        r0, r1, off = int(bt.row_off[b]), int(bt.row_off[b + 1]), int(bt.tok_off[b])
        first = lens[b] - rows[b]
        t = torch.cat([torch.arange(8), torch.randint(0, lens[b], (40,), generator=g), torch.arange(lens[b] - 8, lens[b])])
        rows_of = bt.cache_row(b, t)
        t, rows_of = t[rows_of >= 0], rows_of[rows_of >= 0]
        q, k = bt.q[r0:r1].to(dev).double(), bt.kv[rows_of].to(dev).double()
        w = torch.exp(bt.scale * (q.view(-1, 576) @ k.T).view(r1 - r0, heads, -1) - lse[r0:r1].to(dev).double()[..., None])
        see = t.to(dev)[None, :] <= first + torch.arange(r1 - r0, device=dev)[:, None]
        want = (w * see[:, None, :]).sum((0, 1)).cpu()
        # (0.5 * mass is taken off again: two roundings of the sum)
        assert torch.all((got[off + t] - want).abs() <= 1e-5 * want + 2.0 ** -23 * (want + mass[off + t].double())), b


@pytest.mark.parametrize("lazy", [False, True])
def test_victims_of_caches_with_more_slots_than_a_block_keeps_keys_of(lazy):
    # 10 requests of 524288 slots: 65536 slots a block, of which it keeps 53248 keys and gathers the others again
    B, C, length = 10, 524288, 600_000
    g = torch.Generator(device=dev).manual_seed(8)
    off = torch.arange(B + 1, device=dev) * length
    s2t = torch.stack([torch.randperm(length, generator=g, device=dev)[:C] for _ in range(B)]).to(torch.int32)
    s2t[:, ::41] = -1
    mass = torch.rand(B * length, generator=g, device=dev)
    mass[::3] = 0.25                                        # ties
    mass[1::3] = (mass[1::3] * 8).floor() / 8
    free = torch.zeros((B, C), dtype=torch.bool, device=dev)
    bits = None
    if lazy:
        free = torch.rand((B, C), generator=g, device=dev) < 0.4
        bits = (free.view(B, C // 32, 32).long() << torch.arange(32, device=dev)).sum(2)
        bits = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32).flatten()
    et = torch.empty((B, C), dtype=torch.int32, device=dev)
    es, ec, st = torch.empty_like(et), torch.empty(B, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    for keep in (C // 8, C // 2 + 77):
        L.evict_select(off, B * length, s2t, mass, keep, et, es, ec, st, sinks=100, recent=1000, freebits=bits)
        assert int(st.item()) == 0
        for b in range(B):
            tok = torch.where(free[b], -1, s2t[b]).cpu().numpy()
            slots = np.nonzero(tok >= 0)[0]
            may = slots[(tok[slots] >= 100) & (tok[slots] < length - 1000)]
            want = max(0, min(len(slots) - keep, len(may)))
            m = mass[b * length:(b + 1) * length].cpu().numpy()[tok[may]]
            gone = np.sort(may[np.lexsort((tok[may], m))[:want]])
            assert int(ec[b]) == want > 0 or (want == 0 and int(ec[b]) == 0)
            assert np.array_equal(es[b].cpu().numpy(), np.concatenate([gone, np.full(C - want, -1)]))
            assert np.array_equal(et[b].cpu().numpy(), np.concatenate([tok[gone], np.full(C - want, -1)]))


def test_the_bench_weighs_with_the_lse_of_its_rows():
    import json
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "bench.py", "--part", "paged", "--steps", "2", "--warmup", "3"], cwd=root,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    line = json.loads(r.stdout.strip().splitlines()[-1])
    assert line["status"] == 0 and len(line["weights_per_row_and_head"]) == 2
    assert all(abs(x - 1.0) < 1e-4 for x in line["weights_per_row_and_head"])


# ---------------------------------------------------------------- captured, empty, and first calls
def test_weights_victims_and_release_in_a_replayed_graph():
    # one graph of a step's calls, the weights' workspace taken while it is captured, replayed over growing contexts
    B, n, C = 2, 300, 64
    g = torch.Generator().manual_seed(4)
    host = torch.randn((B * n, 576), generator=g).to(torch.bfloat16).pin_memory()
    off = torch.arange(B + 1, device=dev) * n
    q = torch.randn((B, 128, 576), generator=g).to(torch.bfloat16).to(dev)
    row_off = torch.arange(B + 1, device=dev)

    def state():
        cache = L.LayerCache(B, B * n, C, host)
        end = off[:-1] + 200
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        sel = torch.stack([torch.arange(b, 2 * C, 2) for b in range(B)]).to(torch.int32).to(dev)
        L.cache_step(off, B * n, sel, cache, torch.empty((B, C), dtype=torch.int32, device=dev), st, tok_end=end)
        i = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=dev)
        return dict(cache=cache, end=end, st=st, mass=torch.zeros(B * n, device=dev), et=i(B, C), es=i(B, C), ec=i(B),
                    lse=torch.zeros((B, 128), device=dev), out=torch.zeros((B, 128, 512), dtype=torch.bfloat16, device=dev),
                    ws=torch.empty(L.mla_chunk_workspace_size(B, 128, B), dtype=torch.uint8, device=dev),
                    pages=L.KVPages.of_cache(cache))

    def step(s):
        L.mla_chunk(row_off, q, off, B * n, s["pages"], 0.07, s["out"], s["lse"], s["ws"], s["st"], tok_end=s["end"])
        L.mla_mass(row_off, q, s["lse"], off, B * n, s["pages"], 0.07, s["mass"], s["mass"], s["st"], decay=0.9, tok_end=s["end"])
        L.evict_select(off, B * n, s["cache"].slot2tok, s["mass"], 10, s["et"], s["es"], s["ec"], s["st"], sinks=2, recent=3,
                       tok_end=s["end"], freebits=s["cache"].freebits)
        L.cache_release(off, B * n, s["et"], s["cache"], s["st"], mass=s["mass"], tok_end=s["end"])
        s["end"] += 1
    a, b = state(), state()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=dev) for _ in range(8)]  # not in the graph's pool
    for _ in range(3):
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        for k in ("mass", "et", "es", "ec", "lse", "end"):
            assert torch.equal(a[k], b[k]), k
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["cache"].slot2tok, b["cache"].slot2tok)
        assert int(a["st"].item()) == 0 and int(b["st"].item()) == 0
    assert int((a["cache"].slot2tok >= 0).sum()) == 2 * 10 and len(junk) == 8


def test_calls_without_rows_or_tokens():
    off, st = torch.tensor([0, 40, 90], device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    pages = L.KVPages(torch.arange(6, dtype=torch.int32, device=dev), torch.ones((96, 576), dtype=torch.bfloat16, device=dev), 16)
    none = torch.zeros(3, dtype=torch.int64, device=dev)
    q, lse = torch.empty((0, 16, 576), dtype=torch.bfloat16, device=dev), torch.empty((0, 16), device=dev)
    mass = torch.rand(90, device=dev)
    out = torch.full((90,), 5.0, device=dev)
    L.mla_mass(none, q, lse, off, 90, pages, 0.1, mass, out, st, decay=0.5, tok_end=torch.tensor([30, 90], device=dev))
    want = mass * 0.5
    want[30:40] = 5.0
    assert torch.equal(out, want) and int(st.item()) == 0
    ws = torch.empty(L.mla_chunk_workspace_size(0, 16, 2), dtype=torch.uint8, device=dev)
    L.mla_chunk(none, q, off, 90, pages, 0.1, torch.empty((0, 16, 512), dtype=torch.bfloat16, device=dev), lse, ws, st)
    # requests without tokens: nothing to weigh or to evict
    zero, empty = torch.zeros(3, dtype=torch.int64, device=dev), torch.empty(0, device=dev)
    L.mla_mass(none, q, lse, zero, 0, L.KVPages(torch.empty(0, dtype=torch.int32, device=dev), pages.kv, 16), 0.1, empty, empty, st)
    i = torch.full((2, 32), 3, dtype=torch.int32, device=dev)
    cnt = torch.full((2,), 3, dtype=torch.int32, device=dev)
    L.evict_select(zero, 0, torch.full_like(i, -1), empty, 0, i, i.clone(), cnt, st)
    assert torch.all(i == -1) and torch.all(cnt == 0) and int(st.item()) == 0


def test_a_process_may_capture_its_first_call():
    import subprocess
    import sys
    code = """
import torch
from sparse_attention_kv_echo_gb300 import _lib as L
dev = "cuda"
L.load()
off, rows = torch.tensor([0, 500], device=dev), torch.tensor([0, 40], device=dev)
q = torch.randn((40, 128, 576), device=dev).to(torch.bfloat16)
pages = L.KVPages(torch.arange(32, dtype=torch.int32, device=dev), torch.randn((512, 576), device=dev).to(torch.bfloat16), 16)
out, lse = torch.zeros((40, 128, 512), dtype=torch.bfloat16, device=dev), torch.zeros((40, 128), device=dev)
ws = torch.zeros(L.mla_chunk_workspace_size(40, 128, 1), dtype=torch.uint8, device=dev)
mass, st = torch.zeros(500, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
s2t = torch.arange(64, dtype=torch.int32, device=dev)[None].contiguous()
et, es, ec = torch.zeros_like(s2t), torch.zeros_like(s2t), torch.zeros(1, dtype=torch.int32, device=dev)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    L.mla_chunk(rows, q, off, 500, pages, 0.07, out, lse, ws, st)
    L.mla_mass(rows, q, lse, off, 500, pages, 0.07, mass, mass, st, decay=0.0)
    L.evict_select(off, 500, s2t, mass, 10, et, es, ec, st)
g.replay()
torch.cuda.synchronize()
assert int(st.item()) == 0 and int(ec.item()) == 54 and abs(float(mass.sum()) - 40 * 128) < 1, (st, ec, mass.sum())
print("captured")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-1500:]
