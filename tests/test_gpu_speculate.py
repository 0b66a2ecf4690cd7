"""Steps of speculative decoding as a server runs them, over one pool of pages: a prompt forked into samples, trees reserved,
their rows written, attended in every layer, verified, kept and their pages given up, and the pool closed up between."""
import os
import subprocess
import sys

import pytest
import torch

from _paged import lse_tolerance, out_tolerance
from _speculate import Pool, TreeBatch, ancestors, random_parents, verify

pytestmark = pytest.mark.gpu


def _lib():
    from sparse_attention_kv_echo_gb300 import lib
    return lib


@pytest.mark.parametrize("page,heads,mode", [(16, 16, "sample"), (4, 128, "greedy"), (7, 40, "certain")])
def test_steps(page, heads, mode):
    L, dev = _lib(), "cuda"
    g = torch.Generator().manual_seed(page)
    B, layers, V, region = 4, 2, 50, -(-150 // page) * page
    n_pages = 4 * region // page
    off = [b * region for b in range(B + 1)]
    tokens = off[-1]
    entries = tokens // page
    plain = Pool(entries, n_pages, page, torch.zeros((layers, n_pages * page, 576), dtype=torch.bfloat16))
    i32, i64 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.int64, device=dev)
    pool = L.PagePool(torch.full((entries,), -1, **i32), torch.zeros(n_pages, **i32), plain.kv.to(dev), page)
    ws = torch.empty(L.pages_workspace_size(B, n_pages), dtype=torch.uint8, device=dev)
    status, tok_off = torch.zeros(1, **i32), torch.tensor(off, **i64)
    end, room, new_end = torch.tensor(off[:-1], **i64), torch.zeros(B, **i64), torch.zeros(B, **i64)
    p_end = list(off[:-1])

    def write(b, first, rows):  # the model's new rows of request b's tokens from `first` on: [layers, n, 576]
        for i in range(rows.shape[1]):
            t = off[b] + first + i
            at = plain.tab[t // page] * page + t % page
            plain.kv[:, at] = rows[:, i]
            pool.kv[:, at] = rows[:, i].to(dev)

    def grow(lengths):
        want = [off[b] + n for b, n in enumerate(lengths)]
        L.pages_reserve(tok_off, end, torch.tensor(want, **i64), tokens, pool, room, ws, status)
        got = plain.reserve(off, p_end, want, tokens)
        assert got == want == room.tolist()
        for b in range(B):
            a, z = p_end[b] - off[b], want[b] - off[b]
            if z > a:
                write(b, a, torch.randn((layers, z - a, 576), generator=g).to(torch.bfloat16))
        p_end[:] = want
        end.copy_(room)

    grow([61, 0, 0, 23])                                              # two prompts; then the first one's samples
    L.pages_fork(torch.tensor([0, 0], **i32), torch.tensor([1, 2], **i32), tok_off, end, tokens, pool, ws, status)
    plain.fork([0, 0], [1, 2], off, p_end, tokens)
    for step in range(4):
        rows = [int(torch.randint(1, 9, (1,), generator=g)) for _ in range(B)]
        parents = [random_parents(n, g, 3) for n in rows]
        flat = [p for ps in parents for p in ps]
        grow([e - o + n for e, o, n in zip(p_end, off, rows)])
        lens = [e - o for e, o in zip(p_end, off)]
        n, row_off = sum(rows), torch.tensor([0] + rows).cumsum(0)
        d_row_off, parent = row_off.to(dev), torch.tensor(flat, **i32)
        mask = torch.zeros((n, 1), **i32)
        L.tree_masks(d_row_off, parent, mask, status)
        bt = TreeBatch(lens, rows, [ancestors(p) for p in parents], heads=heads, page=page, seed=step)
        bt.tok_off, bt.tok_end, bt.n_tokens = torch.tensor(off), torch.tensor(p_end), tokens
        bt.tab = torch.tensor(plain.tab, dtype=torch.int32)
        at_ws = torch.empty(L.mla_chunk_workspace_size(n, heads, B), dtype=torch.uint8, device=dev)
        for layer in range(layers):
            out = torch.empty((n, heads, 512), dtype=torch.bfloat16, device=dev)
            lse = torch.empty((n, heads), device=dev)
            L.mla_tree(d_row_off, bt.q.to(dev), mask, tok_off, tokens, pool.of_layer(layer), bt.scale, out, lse, at_ws, status, tok_end=end)
            bt.kv = plain.kv[layer]
            ref, rl, absv, dots = bt.attend()
            assert ((lse.cpu().double() - rl).abs() <= lse_tolerance(dots, rl, max(lens))).all()
            assert ((out.cpu().double() - ref).abs() <= out_tolerance(ref, absv, dots, max(lens))).all()
        logits = 2 * torch.randn((n, V), generator=g)
        target = logits if mode == "greedy" else torch.softmax(logits, -1)
        draft = torch.softmax(logits + 0.5 * torch.randn((n, V), generator=g), -1)
        token = [int(torch.multinomial(draft[int(row_off[b]) + max(p, 0)], 1, generator=g)) if mode == "sample"
                 else int(draft[int(row_off[b]) + max(p, 0)].argmax()) for b, ps in enumerate(parents) for p in ps]
        u_node, u_pick = (None, None) if mode == "greedy" else (torch.rand(n, generator=g), torch.rand(B, generator=g))
        draft = draft if mode == "sample" else None
        put = lambda t: None if t is None else t.to(dev)  # noqa: E731
        path, count, behind = torch.zeros(n, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32)
        L.draft_verify(d_row_off, parent, torch.tensor(token, **i32), target.to(dev), path, count, behind, status, draft=put(draft),
                       u_node=put(u_node), u_pick=put(u_pick))
        L.rows_keep(d_row_off, path, count, tok_off, end, tokens, pool, new_end, status)
        L.pages_free(tok_off, new_end, tokens, pool, status)
        want_path, want_count = [], []
        for b in range(B):
            r0, r1 = int(row_off[b]), int(row_off[b + 1])
            cut = lambda t: None if t is None else t[r0:r1]  # noqa: E731
            p, y = verify(parents[b], token[r0:r1], target[r0:r1], cut(draft), cut(u_node), None if u_pick is None else float(u_pick[b]))
            assert int(behind[b]) == y
            want_path += p + [-1] * (rows[b] - len(p))
            want_count.append(len(p))
        assert path.tolist() == want_path and count.tolist() == want_count
        p_end[:] = plain.keep(row_off.tolist(), want_path, want_count, off, p_end, tokens)
        plain.free(off, p_end, tokens)
        assert new_end.tolist() == p_end
        end.copy_(new_end)
        if step == 1:                                                 # a sample ends; the pool closes up
            p_end[1] = off[1]
            end[1] = off[1]
            plain.free(off, p_end, tokens)
            L.pages_free(tok_off, end, tokens, pool, status)
            used = torch.zeros(1, **i32)
            L.pages_compact(tokens, pool, used, ws, status)
            assert int(used) == plain.compact()
        assert pool.page_tab.tolist() == plain.tab and pool.refs.tolist() == plain.refs
        assert torch.equal(pool.kv.cpu().view(torch.int16), plain.kv.view(torch.int16))
        assert int(status) == 0 and not plain.bad and not plain.full


FIRST_CALL = """
import torch
from sparse_attention_kv_echo_gb300 import lib as L
dev = "cuda"
i32, i64 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.int64, device=dev)
row_off, parent = torch.tensor([0, 3], **i64), torch.tensor([-1, 0, 0], **i32)
tab, refs = torch.full((8,), -1, **i32), torch.zeros(8, **i32)
kv = torch.randn((8 * 16, 576), device=dev).bfloat16()
pool = L.PagePool(tab, refs, kv, 16)
off, end = torch.tensor([0, 64, 128], **i64), torch.tensor([20, 64], **i64)
want = torch.tensor([23, 64], **i64)
q = torch.randn((3, 16, 576), device=dev).bfloat16()
mask, status = torch.zeros((3, 1), **i32), torch.zeros(1, **i32)
out, lse = torch.zeros((3, 16, 512), dtype=torch.bfloat16, device=dev), torch.zeros((3, 16), device=dev)
ws = torch.zeros(L.pages_workspace_size(2, 8), dtype=torch.uint8, device=dev)
aws = torch.zeros(L.mla_chunk_workspace_size(3, 16, 1), dtype=torch.uint8, device=dev)
p = torch.softmax(torch.randn((3, 100), device=dev), -1)
path, count, nxt, new_end = torch.zeros(3, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32), torch.zeros(2, **i64)
u, up, used = torch.rand(3, device=dev), torch.rand(1, device=dev), torch.zeros(1, **i32)
src, dst, zero = torch.tensor([0], **i32), torch.tensor([1], **i32), torch.tensor([0, 64], **i64)
token, rows2, cnt2 = torch.tensor([0, 5, 7], **i32), torch.tensor([0, 3, 3], **i64), torch.zeros(2, **i32)
pages = pool.of_layer()
torch.cuda.synchronize()
s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
    L.pages_reserve(off, zero, want, 128, pool, None, ws, status)
    L.tree_masks(row_off, parent, mask, status)
    L.mla_tree(row_off, q, mask, off[:2], 64, pages, 0.07, out, lse, aws, status, tok_end=want[:1])
    L.draft_verify(row_off, parent, token, p, path, count, nxt, status, draft=p, u_node=u, u_pick=up)
    L.draft_verify(row_off, parent, token, p.bfloat16(), path, count, nxt, status)
    cnt2[:1].copy_(count)
    L.rows_keep(rows2, path, cnt2, off, want, 128, pool, new_end, status)
    L.pages_free(off, new_end, 128, pool, status)
    L.pages_fork(src, dst, off, new_end, 128, pool, ws, status)
    L.pages_compact(128, pool, used, ws, status)
for _ in range(2):
    tab.fill_(-1)
    refs.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert int(status) == 0 and int(used) == len({x for x in tab.tolist() if x >= 0}) > 0, (status, used, tab)
    assert torch.isfinite(lse).all() and 1 <= int(count) <= 3
"""


def test_a_process_may_capture_its_first_calls():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stdout + r.stderr
