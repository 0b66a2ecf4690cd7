"""Calls of speculative decoding on two streams at once, each with a workspace and results of its own, give what they give alone."""
import pytest
import torch

from _speculate import TreeBatch, ancestors, random_parents

pytestmark = pytest.mark.gpu
dev = "cuda"


def _lib():
    from sparse_attention_kv_echo_gb300 import lib
    return lib


class Step:
    """Masks, attention, greedy and sampled verification, and a pool that reserves, keeps and closes up."""

    def __init__(self, lens, rows, heads, vocab, seed):
        L, g = _lib(), torch.Generator().manual_seed(seed)
        parents = [random_parents(n, g, 3) for n in rows]
        self.bt = bt = TreeBatch(lens, rows, [ancestors(p) for p in parents], heads=heads, page=16, seed=seed)
        self.row_off, self.q, self.tok_off, self.end, self.pages = bt.on(dev, L)
        i32 = dict(dtype=torch.int32, device=dev)
        n, B = bt.n, len(lens)
        self.parent = torch.tensor([p for ps in parents for p in ps], **i32)
        self.token = torch.randint(0, vocab, (n,), generator=g).to(torch.int32).to(dev)
        self.target = torch.softmax(2 * torch.randn((n, vocab), generator=g), 1).to(dev)
        self.draft = torch.softmax(2 * torch.randn((n, vocab), generator=g), 1).to(dev)
        self.u, self.pick = torch.rand(n, generator=g).to(dev), torch.rand(B, generator=g).to(dev)
        self.ws = torch.empty(L.mla_chunk_workspace_size(n, heads, B), dtype=torch.uint8, device=dev)
        self.words = -(-max(rows) // 32)
        self.n_pages = 3 * sum(-(-x // 16) for x in lens)
        self.pws = torch.empty(L.pages_workspace_size(B, self.n_pages), dtype=torch.uint8, device=dev)
        region = 16 * (-(-max(lens) // 16) + 4)
        self.off = torch.arange(B + 1, device=dev) * region
        self.want = self.off[:-1] + torch.tensor(lens, device=dev)
        self.rows_kv = torch.randn((2, self.n_pages * 16, 576), generator=g).to(torch.bfloat16).to(dev)
        self.region = region

    def outputs(self):
        bt, i32 = self.bt, dict(dtype=torch.int32, device=dev)
        n, B = bt.n, len(bt.lens)
        z = lambda *s, **k: torch.zeros(s, device=dev, **k)  # noqa: E731
        entries = B * self.region // 16
        return {"mask": z(n, self.words, dtype=torch.int32), "out": z(n, bt.heads, 512, dtype=torch.bfloat16), "lse": z(n, bt.heads),
                "path": z(n, dtype=torch.int32), "count": z(B, dtype=torch.int32), "next": z(B, dtype=torch.int32),
                "path_g": z(n, dtype=torch.int32), "count_g": z(B, dtype=torch.int32), "next_g": z(B, dtype=torch.int32),
                "tab": torch.full((entries,), -1, **i32), "refs": z(self.n_pages, dtype=torch.int32), "kv": self.rows_kv.clone(),
                "new_end": z(B, dtype=torch.int64), "used": z(1, dtype=torch.int32), "status": z(1, dtype=torch.int32)}

    def run(self, o, stream):
        L, bt, st, kw = _lib(), self.bt, o["status"], dict(stream=stream)
        tokens = len(bt.lens) * self.region
        L.tree_masks(self.row_off, self.parent, o["mask"], st, **kw)
        L.mla_tree(self.row_off, self.q, o["mask"], self.tok_off, bt.n_tokens, self.pages, bt.scale, o["out"], o["lse"], self.ws, st,
                   tok_end=self.end, **kw)
        L.draft_verify(self.row_off, self.parent, self.token, self.target, o["path"], o["count"], o["next"], st, draft=self.draft,
                       u_node=self.u, u_pick=self.pick, **kw)
        L.draft_verify(self.row_off, self.parent, self.token, self.target, o["path_g"], o["count_g"], o["next_g"], st, **kw)
        pool = L.PagePool(o["tab"], o["refs"], o["kv"], 16)
        L.pages_reserve(self.off, self.off[:-1].contiguous(), self.want, tokens, pool, None, self.pws, st, **kw)
        L.rows_keep(self.row_off, o["path"], o["count"], self.off, self.want, tokens, pool, o["new_end"], st, **kw)
        L.pages_free(self.off, o["new_end"], tokens, pool, st, **kw)
        L.pages_compact(tokens, pool, o["used"], self.pws, st, **kw)


def test_two_streams_at_once():
    steps = [Step([700, 90, 1500], [7, 40, 2], 128, 5003, 1), Step([260] * 24, [5] * 24, 16, 20011, 2)]
    alone = []
    main = torch.cuda.current_stream()
    for s in steps:
        o = s.outputs()
        s.run(o, main)
        torch.cuda.synchronize()
        assert int(o["status"]) == 0
        alone.append(o)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    many = [[s.outputs() for _ in range(12)] for s in steps]
    for st in streams:
        st.wait_stream(main)
    for i in range(12):
        for k, s in enumerate(steps):
            s.run(many[k][i], streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        for o in many[k]:
            for name, x in alone[k].items():
                assert torch.equal(x.view(torch.uint8), o[name].view(torch.uint8)), name
