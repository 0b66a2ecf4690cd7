"""Speculative decoding where offsets pass 32 bits: caches, pools and rows of probabilities of more than 4 GB."""
import pytest
import torch

from _paged import lse_tolerance, out_tolerance
from _speculate import TreeBatch, ancestors, verify

pytestmark = pytest.mark.gpu


def _lib():
    from sparse_attention_kv_echo_gb300 import lib
    return lib


def test_trees_over_pages_behind_four_gigabytes():
    L, dev = _lib(), "cuda"
    page, far = 16, 4_000_000 // 16                      # the pages lie from 4.6 GB on
    bt = TreeBatch([300, 77], [9, 5], [ancestors([-1, 0, 0, 1, 2, 2, 4, 3, 0]), ancestors([-1, 0, 0, 2, 1])], heads=16,
                   page=page, seed=3)
    row_off, q, tok_off, end, _ = bt.on(dev, L)
    kv = torch.empty((far * page + bt.kv.shape[0], 576), dtype=torch.bfloat16, device=dev)
    kv[far * page:] = bt.kv.to(dev)
    pages = L.KVPages((bt.tab + far).to(dev), kv, page)
    out = torch.empty((bt.n, 16, 512), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((bt.n, 16), device=dev)
    ws = torch.empty(L.mla_chunk_workspace_size(bt.n, 16, 2), dtype=torch.uint8, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    L.mla_tree(row_off, q, bt.mask(1).to(dev), tok_off, bt.n_tokens, pages, bt.scale, out, lse, ws, status, tok_end=end)
    ref, rl, absv, dots = bt.attend()
    assert int(status) == 0
    assert ((lse.cpu().double() - rl).abs() <= lse_tolerance(dots, rl, 300)).all()
    assert ((out.cpu().double() - ref).abs() <= out_tolerance(ref, absv, dots, 300)).all()


def test_pages_of_a_pool_behind_four_gigabytes():
    # two layers of 5.2 GB each; what is used lies at the pool's end
    L, dev, page, n_pages = _lib(), "cuda", 64, 70_000
    g = torch.Generator(device=dev).manual_seed(1)
    kv = torch.zeros((2, n_pages * page, 576), dtype=torch.bfloat16, device=dev)
    i32, i64 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.int64, device=dev)
    tab = torch.full((8,), -1, **i32)                      # two requests of four pages each
    tab[0], tab[1] = n_pages - 1, n_pages - 4
    refs = torch.zeros(n_pages, **i32)
    refs[n_pages - 1] = refs[n_pages - 4] = 1
    pool = L.PagePool(tab, refs, kv, page)
    rows = torch.randn((2, 100, 576), generator=g, device=dev).to(torch.bfloat16)   # the request's 100 tokens

    def place(p, n):
        return kv[:, p * page:p * page + n]

    def content(pages):
        return torch.cat([place(p, min(page, 100 - page * i)) for i, p in enumerate(pages)], 1)

    place(n_pages - 1, 64)[:] = rows[:, :64]
    place(n_pages - 4, 36)[:] = rows[:, 64:]
    off, end = torch.tensor([0, 256, 512], **i64), torch.tensor([100, 256], **i64)
    ws = torch.empty(L.pages_workspace_size(2, n_pages), dtype=torch.uint8, device=dev)
    status = torch.zeros(1, **i32)
    # the last rows' page is copied to the lowest free one, page 0
    L.pages_fork(torch.tensor([0], **i32), torch.tensor([1], **i32), off, end, 512, pool, ws, status)
    assert tab.tolist() == [n_pages - 1, n_pages - 4, -1, -1, n_pages - 1, 0, -1, -1] and end.tolist() == [100, 356]
    assert torch.equal(content([n_pages - 1, 0]), rows)
    # a tree of the last five rows of request 0, nodes 0, 2 and 4 accepted: within a far page
    new_end = torch.empty(2, **i64)
    L.rows_keep(torch.tensor([0, 5, 5], **i64), torch.tensor([0, 2, 4, -1, -1], **i32), torch.tensor([3, 0], **i32), off, end, 512,
                pool, new_end, status)
    assert new_end.tolist() == [98, 356]
    assert torch.equal(place(n_pages - 4, 34), rows[:, [*range(64, 96), 97, 99]])
    # both requests grow; three pages in use move to the first places
    L.pages_reserve(off, torch.tensor([98, 356], **i64), torch.tensor([130, 356], **i64), 512, pool, None, ws, status)
    assert tab.tolist() == [n_pages - 1, n_pages - 4, 1, -1, n_pages - 1, 0, -1, -1]
    used = torch.empty(1, **i32)
    L.pages_compact(512, pool, used, ws, status)
    assert int(used) == 4 and int(status) == 0
    assert tab.tolist() == [3, 2, 1, -1, 3, 0, -1, -1]
    assert refs[:4].tolist() == [1, 1, 1, 2] and int(refs.sum()) == 5
    assert torch.equal(content([3, 0]), rows)
    assert torch.equal(place(2, 34), rows[:, [*range(64, 96), 97, 99]])


@pytest.mark.parametrize("mode", ["sample", "greedy"])
def test_rows_of_probabilities_behind_four_gigabytes(mode):
    # three rows of 2^24 tokens behind 2^31 of other requests'
    L, dev, V, first = _lib(), "cuda", 1 << 24, 128
    g = torch.Generator(device=dev).manual_seed(7)
    n = first + 3
    target = torch.zeros((n, V), dtype=torch.bfloat16, device=dev)
    some = torch.randint(0, V, (3, 4000), generator=g, device=dev)
    w = torch.softmax(torch.randn((3, 4000), generator=g, device=dev), 1).to(torch.bfloat16)
    target[first:].scatter_(1, some, w)
    draft = None
    if mode == "sample":
        draft = torch.zeros((n, V), dtype=torch.bfloat16, device=dev)
        draft[first:].scatter_(1, some, w.flip(1))
    tokens = [0, int(some[0, w[0].argmax()]), int(some[1, 17])]
    i32 = dict(dtype=torch.int32, device=dev)
    parent, token = torch.full((n,), -1, **i32), torch.zeros(n, **i32)
    parent[first + 1], parent[first + 2] = 0, 1
    token[first:] = torch.tensor(tokens, **i32)
    u, pick = torch.full((n,), 0.9, device=dev), torch.full((1,), 0.75, device=dev)
    path, count, behind = torch.full((n,), 9, **i32), torch.full((1,), 9, **i32), torch.full((1,), 9, **i32)
    status = torch.zeros(1, **i32)
    kw = dict(draft=draft, u_node=u, u_pick=pick) if mode == "sample" else {}
    L.draft_verify(torch.tensor([first, n], dtype=torch.int64, device=dev), parent, token, target, path, count, behind, status, **kw)
    rows = target[first:].cpu()
    if mode == "sample":
        want, y = verify([-1, 0, 1], tokens, rows, draft[first:].cpu(), [0.9] * 3, 0.75)
    else:
        want, y = verify([-1, 0, 1], tokens, rows, None, None, None)
    assert (path[:first] == 9).all() and int(status) == 0
    assert path[first:].tolist() == want + [-1] * (3 - len(want))
    assert (int(count), int(behind)) == (len(want), y)
