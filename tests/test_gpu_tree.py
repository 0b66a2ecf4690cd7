"""echo_tree_masks and echo_mla_tree against their plain forms."""
import pytest
import torch

from _paged import lse_tolerance, out_tolerance
from _speculate import TreeBatch, ancestors, mask_words, random_parents

pytestmark = pytest.mark.gpu


def _lib():
    from sparse_attention_kv_echo_gb300 import lib
    return lib


def _masks(rows, parents, words, dev="cuda", spare=0):
    L = _lib()
    n = sum(rows)
    off = torch.tensor([0] + rows, dtype=torch.int64).cumsum(0).to(dev)
    parent = torch.tensor([p for ps in parents for p in ps] + [0] * spare, dtype=torch.int32, device=dev)
    mask = torch.full((n + spare, words), 77, dtype=torch.int32, device=dev)
    depth = torch.full((n + spare,), 78, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    L.tree_masks(off, parent, mask, status, depth=depth)
    return mask.cpu(), depth.cpu(), int(status)


@pytest.mark.parametrize("rows,words,reach", [([1], 1, 1), ([5], 1, 1), ([0, 3, 0, 7], 1, 4), ([32, 33], 2, 3), ([64], 2, 1),
                                              ([100, 1, 65], 4, 10), ([1024], 32, 1), ([1000, 17], 32, 7), ([300], 32, 300)])
def test_masks_are_the_ancestors(rows, words, reach):
    g = torch.Generator().manual_seed(sum(rows))
    parents = [random_parents(n, g, reach) for n in rows]
    mask, depth, status = _masks(rows, parents, words, spare=2)
    n = sum(rows)
    sets = [s for ps in parents for s in ancestors(ps)]
    assert torch.equal(mask[:n], mask_words(sets, words)) and status == 0
    assert depth[:n].tolist() == [len(s) - 1 for s in sets]
    assert (mask[n:] == 77).all() and (depth[n:] == 78).all()          # rows of no request


def test_forests_bad_parents_and_trees_too_large():
    L = _lib()
    mask, depth, status = _masks([6], [[-1, -1, 0, 1, -1, 4]], 1)
    assert mask[:, 0].tolist() == [1, 2, 5, 10, 16, 48] and depth.tolist() == [0, 0, 1, 1, 0, 1] and status == 0
    mask, depth, status = _masks([5], [[3, 1, 0, -7, 2 ** 30]], 1)     # each counts as none
    assert mask[:, 0].tolist() == [1, 2, 5, 8, 16] and status == L.ST_BADDATA
    mask, depth, status = _masks([33, 2], [[-1] + list(range(32)), [-1, 0]], 1)
    assert (mask[:33] == 0).all() and (depth[:33] == 0).all() and mask[33:, 0].tolist() == [1, 3]
    assert status == L.ST_BADDATA


def _attend(bt, words=None, mask=None, tok_end=True, stream=None):
    L = _lib()
    dev = "cuda"
    row_off, q, tok_off, end, pages = bt.on(dev, L)
    words = words or -(-max(max(bt.rows), 1) // 32)
    mask = (bt.mask(words) if mask is None else mask).to(dev)
    out = torch.full((bt.n, bt.heads, 512), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((bt.n, bt.heads), 7.0, device=dev)
    ws = torch.full((L.mla_chunk_workspace_size(bt.n, bt.heads, len(bt.lens)),), 255, dtype=torch.uint8, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    L.mla_tree(row_off, q, mask, tok_off, bt.n_tokens, pages, bt.scale, out, lse, ws, status, tok_end=end, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), int(status)


def _compare(bt, out, lse):
    ref, rl, absv, dots = bt.attend()
    none = torch.isinf(rl)
    n = max(bt.lens)
    assert (torch.isinf(lse) == none).all() and (out[none] == 0).all()
    err = (lse.double() - rl).abs().nan_to_num(0.0, 0.0, 0.0)
    assert (err <= lse_tolerance(dots, rl, n)).all(), err.max()
    off = (out.double() - ref).abs()
    assert (off <= out_tolerance(ref, absv, dots, n)).all(), off.max()


CASES = [  # lens (trees included), nodes, heads, page, reach, absent
    ([1], [1], 128, 16, 1, 0.0), ([9], [9], 128, 4, 3, 0.0), ([70], [6], 128, 64, 2, 0.0), ([200], [40], 16, 48, 5, 0.0),
    ([333], [33], 1, 1, 4, 0.3), ([130, 64, 5], [64, 1, 5], 40, 7, 9, 0.2), ([1500], [4], 128, 64, 2, 0.1),
    ([3000, 900], [20, 70], 16, 256, 30, 0.05), ([257] * 40, [3] * 40, 16, 16, 1, 0.0), ([4100], [130], 8, 64, 6, 0.0),
    ([600, 0, 40], [8, 0, 2], 64, 32, 3, 0.0)]


@pytest.mark.parametrize("lens,rows,heads,page,reach,absent", CASES)
def test_trees(lens, rows, heads, page, reach, absent):
    g = torch.Generator().manual_seed(len(lens) + heads)
    seen = [ancestors(random_parents(n, g, reach)) for n in rows]
    bt = TreeBatch(lens, rows, seen, heads=heads, page=page, seed=heads + page, absent=absent)
    out, lse, status = _attend(bt)
    assert status == 0
    _compare(bt, out, lse)


@pytest.mark.parametrize("lens,rows,heads", [([40], [40], 16), ([64, 31], [33, 31], 128), ([500], [96], 3)])
def test_any_mask_and_rows_that_see_nothing(lens, rows, heads):
    # bits of no kinship, rows without their own bit, rows without any; bits behind the row are ignored
    g = torch.Generator().manual_seed(heads)
    seen, words = [], 4
    mask = torch.randint(-2 ** 31, 2 ** 31, (sum(rows), words), generator=g).to(torch.int32)
    mask[::3] = 0
    mask[1::5] = -1
    at = 0
    for n in rows:
        seen.append([{j for j in range(n) if (int(mask[at + i, j // 32]) >> (j % 32)) & 1} for i in range(n)])
        at += n
    bt = TreeBatch(lens, rows, seen, heads=heads, page=8, seed=1)
    out, lse, status = _attend(bt, words, mask)
    assert status == 0
    _compare(bt, out, lse)
    if lens[0] == rows[0]:
        assert torch.isinf(lse[0]).all()


@pytest.mark.parametrize("absent", [0.0, 0.4])
def test_trees_over_slots_of_each_requests_own(absent):
    # page 1 and rows per request: the slots of a layer's cache
    g = torch.Generator().manual_seed(4)
    rows = [9, 1, 20]
    seen = [ancestors(random_parents(n, g, 4)) for n in rows]
    bt = TreeBatch([100, 30, 61], rows, seen, heads=16, page=1, seed=7, absent=absent, per_request=128)
    out, lse, status = _attend(bt)
    assert status == 0
    _compare(bt, out, lse)


def test_a_chain_is_the_causal_call():
    L = _lib()
    bt = TreeBatch([700, 300], [40, 3], [ancestors([-1] + list(range(39))), ancestors([-1, 0, 1])], heads=128, page=64, seed=3)
    out, lse, _ = _attend(bt)
    row_off, q, tok_off, end, pages = bt.on("cuda", L)
    o2, l2 = torch.empty((bt.n, 128, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((bt.n, 128), device="cuda")
    ws = torch.empty(L.mla_chunk_workspace_size(bt.n, 128, 2), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.mla_chunk(row_off, q, tok_off, bt.n_tokens, pages, bt.scale, o2, l2, ws, status, tok_end=end)
    ref, rl, absv, dots = bt.attend()
    assert ((lse - l2.cpu()).double().abs() <= 2 * lse_tolerance(dots, rl, 700)).all()
    assert ((out.double() - o2.cpu().double()).abs() <= 2 * out_tolerance(ref, absv, dots, 700)).all()


def test_siblings_do_not_see_each_other_whatever_their_rows_hold():
    # a node's cache row may be large; only its own path feels it.  (The others' last bits may change: rows of a warp move
    # the reference of their softmax together, and the weights' rounding to bf16 goes with it.  Both runs are held to the
    # 64-bit form, which does not change for them.)
    parents = [-1, 0, 0, 0, 2]
    bt = TreeBatch([70], [5], [ancestors(parents)], heads=16, page=16, seed=5)
    out, lse, _ = _attend(bt)
    row = int(bt.cache_row(0, torch.tensor([70 - 5 + 1])))
    bt.kv[row] *= 100
    o2, l2, _ = _attend(bt)
    _compare(bt, o2, l2)
    same = [0, 2, 3, 4]
    ref, rl, absv, dots = bt.attend()
    assert ((lse[same].double() - rl[same]).abs() <= lse_tolerance(dots[same], rl[same], 70)).all()
    assert ((out[same].double() - ref[same]).abs() <= out_tolerance(ref, absv, dots, 70)[same]).all()
    assert not torch.equal(lse[1], l2[1])


def test_requests_that_do_not_fit_see_nothing():
    L = _lib()
    seen = [ancestors([-1] + [0] * 39), ancestors([-1, 0])]
    bt = TreeBatch([100, 60], [40, 2], seen, heads=16, page=16, seed=2)
    mask = torch.zeros((42, 1), dtype=torch.int32)
    mask[40:] = mask_words(seen[1], 1)
    out, lse, status = _attend(bt, 1, mask)                            # 40 rows, 32 bits
    assert status == L.ST_BADDATA and torch.isinf(lse[:40]).all() and (out[:40] == 0).all()
    ref, rl, absv, dots = bt.attend()
    assert ((lse[40:].double() - rl[40:]).abs() <= lse_tolerance(dots[40:], rl[40:], 100)).all()


def test_another_stream_and_a_replayed_graph():
    L = _lib()
    g = torch.Generator().manual_seed(9)
    parents = [random_parents(n, g, 3) for n in (12, 5)]
    bt = TreeBatch([400, 90], [12, 5], [ancestors(p) for p in parents], heads=32, page=16, seed=6)
    out, lse, _ = _attend(bt)
    o2, l2, _ = _attend(bt, stream=torch.cuda.Stream())
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    row_off, q, tok_off, end, pages = bt.on("cuda", L)
    parent = torch.tensor([p for ps in parents for p in ps], dtype=torch.int32, device="cuda")
    mask = torch.zeros((17, 1), dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o3, l3 = torch.zeros_like(out, device="cuda"), torch.zeros_like(lse, device="cuda")
    ws = torch.empty(L.mla_chunk_workspace_size(17, 32, 2), dtype=torch.uint8, device="cuda")

    def step():
        L.tree_masks(row_off, parent, mask, status)
        L.mla_tree(row_off, q, mask, tok_off, bt.n_tokens, pages, bt.scale, o3, l3, ws, status, tok_end=end)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
        with torch.cuda.graph(graph, stream=s):
            step()
    o3.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o3.cpu(), out) and torch.equal(l3.cpu(), lse)
    # another tree in the same buffers
    other = [random_parents(n, g, 3) for n in (12, 5)]
    parent.copy_(torch.tensor([p for ps in other for p in ps], dtype=torch.int32))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    bt.seen = [ancestors(p) for p in other]
    _compare(bt, o3.cpu(), l3.cpu())
    assert int(status) == 0


@pytest.mark.slow
def test_a_tree_behind_a_long_context_by_sampled_rows():
    n, m = 60000, 64
    g = torch.Generator().manual_seed(1)
    seen = ancestors(random_parents(m, g, 8))
    bt = TreeBatch([n], [m], [seen], heads=128, page=64, seed=8)
    out, lse, status = _attend(bt)
    assert status == 0
    kv = bt.kv.double()
    for i in (0, 17, 40, 63):
        t = bt.visible(0, i)
        k = kv[bt.cache_row(0, t)]
        s = bt.scale * bt.q[i].double() @ k.T
        rl = torch.logsumexp(s, -1)
        w = torch.exp(s - rl[:, None])
        dots = bt.scale * (bt.q[i].double().abs() @ k.abs().T).amax(-1)
        ref, absv = w @ k[:, :512], w @ k[:, :512].abs()
        assert ((lse[i].double() - rl).abs() <= lse_tolerance(dots, rl, n)).all()
        assert ((out[i].double() - ref).abs() <= out_tolerance(ref, absv, dots, n)).all()
