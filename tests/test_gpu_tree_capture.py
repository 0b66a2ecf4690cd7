"""echo_mla_tree in a captured graph behind whatever comes before it: nothing, a copy, two streams that join, another layer's
call in the same workspace.  Equal inputs give equal bits."""
import pytest
import torch

from _speculate import TreeBatch, ancestors, random_parents

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,rows,heads", [([400, 90], [12, 5], 32), ([260] * 40, [9] * 40, 128)])  # planned by a warp, by a block
def test_what_comes_before_a_captured_call(lens, rows, heads):
    from sparse_attention_kv_echo_gb300 import lib as L
    g, dev = torch.Generator().manual_seed(heads), "cuda"
    bt = TreeBatch(lens, rows, [ancestors(random_parents(n, g, 3)) for n in rows], heads=heads, page=16, seed=1)
    row_off, q, tok_off, end, pages = bt.on(dev, L)
    mask, status = bt.mask(1).to(dev), torch.zeros(1, dtype=torch.int32, device=dev)
    ws = torch.empty(L.mla_chunk_workspace_size(bt.n, heads, len(lens)), dtype=torch.uint8, device=dev)
    qs = [q, torch.randn(q.shape, generator=g).to(torch.bfloat16).to(dev), q.flip(0).contiguous()]

    def outputs():
        return torch.zeros((bt.n, heads, 512), dtype=torch.bfloat16, device=dev), torch.zeros((bt.n, heads), device=dev)

    def attend(q, out, lse):
        L.mla_tree(row_off, q, mask, tok_off, bt.n_tokens, pages, bt.scale, out, lse, ws, status, tok_end=end)
    want = [outputs() for _ in qs]
    for x, o in zip(qs, want):
        attend(x, *o)
    got, copied, late = [outputs() for _ in range(4)], torch.zeros_like(q), torch.zeros_like(mask)
    s, side, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        attend(qs[0], *got[0])                                         # the graph's first
        attend(qs[1], *got[1])                                         # behind another layer's, in its workspace
        copied.copy_(qs[2])
        attend(copied, *got[2])                                        # behind a copy of what it reads
        side.wait_stream(s)
        with torch.cuda.stream(side):
            late.copy_(mask)
        copied.zero_()
        copied.add_(qs[1])
        s.wait_stream(side)
        L.mla_tree(row_off, copied, late, tok_off, bt.n_tokens, pages, bt.scale, *got[3], ws, status, tok_end=end)  # behind both
    for _ in range(5):
        for o in got:
            for t in o:
                t.zero_()
        late.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((0, 1, 2, 3), (0, 1, 2, 1)):
            assert torch.equal(got[a][0], want[b][0]) and torch.equal(got[a][1], want[b][1]), a
    assert int(status) == 0
