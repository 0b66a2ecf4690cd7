"""echo_draft_verify against the definition in 64 bits (whole numbers, which have to be equal).

The call's sums are good to 2^-48 a value, the definition's to 2^-52 of the running sum: a draw or a test falls on
different sides of its border with a chance of vocab * vocab * 2^-48 at the worst, below 1e-4 at 100000 tokens."""
import pytest
import torch

from _speculate import random_parents, verify

pytestmark = pytest.mark.gpu


def _lib():
    from sparse_attention_kv_echo_gb300 import lib
    return lib


class Drafts:
    """Trees of drafts, their probabilities and uniform numbers, on the CPU."""

    def __init__(self, rows, vocab, reach=1, half=False, mode="sample", noise=0.8, sharp=3.0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.vocab, self.mode = rows, vocab, mode
        self.off = torch.tensor([0] + rows, dtype=torch.int64).cumsum(0)
        n = int(self.off[-1])
        dtype = torch.bfloat16 if half else torch.float32
        t = sharp * torch.randn((n, vocab), generator=g)
        d = torch.softmax(t + noise * torch.randn((n, vocab), generator=g), -1)
        self.target = (t if mode == "greedy" else torch.softmax(t, -1)).to(dtype)
        self.draft = d.to(dtype) if mode == "sample" else None
        self.parent, self.token = [], []
        for b, m in enumerate(rows):
            ps = random_parents(m, g, reach)
            self.parent += ps
            for i in range(m):
                row = d[int(self.off[b]) + max(ps[i], 0)]
                if mode == "sample":
                    self.token.append(int(torch.multinomial(row, 1, generator=g)))
                else:
                    best = row.topk(min(3, vocab))[1]
                    self.token.append(int(best[int(torch.randint(0, len(best), (1,), generator=g)) if i % 2 else 0]))
        self.u_node = None if mode == "greedy" else torch.rand(n, generator=g)
        self.u_pick = None if mode == "greedy" else torch.rand(len(rows), generator=g)

    def run(self, **kw):
        L, dev = _lib(), "cuda"
        n, B = len(self.parent), len(self.rows)
        i32 = dict(dtype=torch.int32, device=dev)
        path, count, behind = torch.full((n,), 55, **i32), torch.full((B,), 56, **i32), torch.full((B,), 57, **i32)
        status = torch.zeros(1, **i32)
        put = lambda t: None if t is None else t.to(dev)  # noqa: E731
        L.draft_verify(self.off.to(dev), torch.tensor(self.parent, **i32), torch.tensor(self.token, **i32), put(self.target),
                       path, count, behind, status, draft=put(self.draft), u_node=put(self.u_node), u_pick=put(self.u_pick), **kw)
        torch.cuda.synchronize()
        return path.tolist(), count.tolist(), behind.tolist(), int(status)

    def expected(self):
        paths, counts, picks = [], [], []
        for b, m in enumerate(self.rows):
            r0, r1 = int(self.off[b]), int(self.off[b + 1])
            if m == 0:
                counts.append(0)
                picks.append(-1)
                continue
            cut = lambda t: None if t is None else t[r0:r1]  # noqa: E731
            p, y = verify(self.parent[r0:r1], self.token[r0:r1], self.target[r0:r1], cut(self.draft), cut(self.u_node),
                          None if self.u_pick is None else float(self.u_pick[b]))
            paths += p + [-1] * (m - len(p))
            counts.append(len(p))
            picks.append(y)
        return paths, counts, picks

    def check(self, status=0):
        path, count, behind, st = self.run()
        assert (path, count, behind) == self.expected()
        assert st == status
        return count


@pytest.mark.parametrize("mode", ["sample", "certain", "greedy"])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rows,vocab,reach", [([1], 1, 1), ([1], 2, 1), ([3], 5, 1), ([4, 0, 1], 31, 2), ([7] * 9, 1000, 1),
                                              ([48, 5], 4099, 12), ([5], 32000, 1), ([33] * 3, 777, 33), ([2] * 80, 130, 1)])
def test_walks(rows, vocab, reach, half, mode):
    Drafts(rows, vocab, reach, half, mode, seed=vocab + len(rows)).check()


@pytest.mark.parametrize("mode", ["sample", "certain"])
def test_many_siblings_are_tried_in_turn(mode):
    # drafts far from the target: most are rejected, the residual falls through many sums (S well above 1)
    rejected = 0
    for seed in range(6):
        d = Drafts([60] * 4, 300, 60, mode=mode, noise=4.0, sharp=2.0, seed=seed)
        d.parent = [-1 if i % 60 == 0 else 0 for i in range(240)]
        if mode == "sample":  # all of them drawn from the root's row
            g = torch.Generator().manual_seed(seed)
            for b in range(4):
                d.token[60 * b:60 * b + 60] = torch.multinomial(d.draft[60 * b], 60, replacement=True, generator=g).tolist()
        rejected += sum(c == 1 for c in d.check())
    assert rejected > 0


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("vocab", [8192, 8195, 100003])
def test_rows_on_any_boundary(vocab, half):
    # rows of an odd vocabulary start at every offset of a 16-byte piece
    Drafts([3, 2, 4, 1, 1, 5], vocab, 2, half, seed=vocab).check()
    Drafts([3, 2, 4, 1, 1, 5], vocab, 2, half, "greedy", seed=vocab).check()


def test_a_vocabulary_of_a_million():
    d = Drafts([2, 1], (1 << 20) + 3, seed=1)
    d.check()
    d = Drafts([2, 1], (1 << 20) + 3, mode="greedy", half=True, seed=2)
    d.check()


def test_results_do_not_hang_on_the_batch():
    # 300 requests take one CTA each, one takes a cluster
    d = Drafts([4] * 300, 2000, 2, seed=11)
    path, count, behind, _ = d.run()
    for b in (0, 7, 150, 299):
        one = Drafts([4], 2000, 2, seed=11)
        one.parent, one.token = d.parent[4 * b:4 * b + 4], d.token[4 * b:4 * b + 4]
        one.target, one.draft = d.target[4 * b:4 * b + 4], d.draft[4 * b:4 * b + 4]
        one.u_node, one.u_pick = d.u_node[4 * b:4 * b + 4], d.u_pick[b:b + 1]
        p, c, y, _ = one.run()
        assert (p, c[0], y[0]) == (path[4 * b:4 * b + 4], count[b], behind[b])
    d.check()


def test_equal_distributions_accept_everything():
    d = Drafts([6] * 3, 500, 1, noise=0.0, seed=4)
    d.draft = d.target.clone()
    assert d.check() == [6, 6, 6]


def test_borders():
    d = Drafts([2], 4, seed=0)
    d.parent, d.token = [-1, 0], [2, 1]
    d.target = torch.tensor([[0.0, 0.25, 0.0, 0.75], [0.0, 0.5, 0.5, 0.0]])
    d.draft = torch.tensor([[0.0, 0.5, 0.5, 0.0], [1.0, 0.0, 0.0, 0.0]])
    for un, up, want in ((0.0, 0.0, ([0, 1], 1)), (0.49999997, 0.0, ([0, 1], 1)), (0.5, 0.0, ([0, -1], 3)),     # u q < p
                         (0.25, 0.5, ([0, 1], 2)), (0.25, 0.49999997, ([0, 1], 1)), (0.25, 0.99999994, ([0, 1], 2)),
                         (0.75, 0.99999994, ([0, -1], 3))):
        d.u_node, d.u_pick = torch.tensor([0.9, un]), torch.tensor([up])
        path, count, behind, st = d.run()
        assert (path, behind[0], st) == (want[0], want[1], 0), (un, up)
        d.check()


def test_a_draft_without_probability_and_a_rejection_that_leaves_nothing():
    d = Drafts([3], 4, seed=0)
    d.parent, d.token = [-1, 0, 0], [0, 3, 1]
    d.target = torch.tensor([[0.0, 0.5, 0.5, 0.0]]).repeat(3, 1)
    d.draft = torch.tensor([[0.0, 0.5, 0.5, 0.0]]).repeat(3, 1)
    d.u_node, d.u_pick = torch.tensor([0.0, 0.0, 0.3]), torch.tensor([0.6])
    # token 3 has neither p nor q: rejected, and max(0, p - q) is empty, so node 2 is tried against p itself
    assert d.run()[:3] == ([0, 2, -1], [2], [2])
    d.check()


def test_the_same_token_twice_among_siblings():
    for mode in ("sample", "certain"):
        d = Drafts([4], 6, mode=mode, seed=3)
        d.parent, d.token = [-1, 0, 0, 0], [0, 2, 2, 4]
        d.u_node = torch.tensor([0.0, 0.999, 0.0, 0.9])
        d.check()


def test_values_that_are_no_probabilities():
    L = _lib()
    for bad in (float("nan"), -0.5, 3.0, float("inf")):
        d = Drafts([2, 2], 64, seed=5)
        d.token[1], d.target[0, 20] = 20, 0.0                          # rejected: the rows are read
        d.target[0, 7] = bad
        d.target[0, 8] = -0.0                                          # is 0, and no fault
        path, count, behind, st = d.run()
        fit = Drafts([2, 2], 64, seed=5)
        fit.token[1], fit.target[0, 20] = 20, 0.0
        fit.target[0, 7], fit.target[0, 8] = (2.0 if bad > 2 else 0.0), 0.0
        assert (path, count, behind) == fit.expected() and st == L.ST_NAN
    d = Drafts([1], 9, seed=1)
    d.target[:] = 0
    assert d.run() == ([0], [1], [0], L.ST_BADDATA)
    d = Drafts([3], 50, seed=2)
    e = Drafts([3], 50, seed=2)
    d.u_node, e.u_node = torch.tensor([0.5, 1.5, -1.0]), torch.tensor([0.5, 0.99999994, 0.0])
    d.u_pick, e.u_pick = torch.tensor([float("nan")]), torch.tensor([0.0])
    path, count, behind, st = d.run()
    assert (path, count, behind) == e.expected() and st == L.ST_BADDATA


@pytest.mark.parametrize("half", [False, True])
def test_rows_of_no_probabilities_give_some_token(half):
    # sums far beyond what the call is made for, and beyond 64 bits: a token in range all the same
    L = _lib()
    for value in (1.0, 2.0, 0.01):
        for seed in range(4):
            d = Drafts([3] * 5, 20000, half=half, seed=seed)
            d.target[:] = value
            d.draft[:] = value / 4
            path, count, behind, st = d.run()
            assert all(0 <= y < 20000 for y in behind) and all(1 <= c <= 3 for c in count)
            assert st in (0, L.ST_BADDATA)                             # (a sum may come out as 0 in 64 bits)
    d = Drafts([3] * 5, 20000, half=half, seed=1)
    d.target = (5 * torch.randn((15, 20000))).to(d.target.dtype)       # logits
    path, count, behind, st = d.run()
    assert all(0 <= y < 20000 for y in behind) and st & L.ST_NAN


def test_tokens_and_parents_out_of_range():
    L = _lib()
    d = Drafts([5], 40, 5, seed=8)
    d.parent, d.token = [-1, 0, 0, 7, 2], [0, -3, d.token[2], 1, 40]
    d.u_node[:] = 0.0                                                  # node 2 is accepted, node 4 is not to be
    path, count, behind, st = d.run()
    assert path == [0, 2, -1, -1, -1] and count == [2] and st == L.ST_BADDATA
    e = Drafts([5], 40, 5, seed=8)
    e.parent, e.token, e.u_node = [-1, 0, 0, -1, 2], d.token, d.u_node
    assert e.expected() == (path, count, behind)


def test_greedy_ties_infinities_and_nan():
    L = _lib()
    d = Drafts([3, 1, 2], 1000, 1, mode="greedy", seed=0)
    d.target[:] = -float("inf")
    d.target[0, [400, 90, 999]] = 5.0                                  # three are the largest: the first
    d.target[1, 998] = 2.0
    d.token[1], d.token[2] = 90, 3
    d.check()
    assert d.run()[2][1] == 0                                          # all -inf: the first token
    d.target[4, 5], d.target[4, 6] = float("nan"), 1.0
    path, count, behind, st = d.run()
    assert st == L.ST_NAN and behind[2] == 6 and (path, count, behind) == d.expected()
    d.target[4] = float("nan")
    assert d.run()[2][2] == 0
    d.target[4, 0] = -0.0
    d.target[4, 1] = 0.0                                               # equal to -0
    assert d.run()[2][2] == 0


def test_trees_too_large_and_inconsistent_bounds():
    L = _lib()
    d = Drafts([3], 20, seed=1)
    n = 1030
    d.rows, d.off = [n, 2], torch.tensor([0, n, n + 2])
    d.parent, d.token = [-1] + [0] * (n - 1) + [-1, 0], [1] * (n + 2)
    d.target = torch.softmax(torch.randn((n + 2, 20)), -1)
    d.draft, d.u_node, d.u_pick = d.target.clone(), torch.zeros(n + 2), torch.tensor([0.5, 0.5])
    path, count, behind, st = d.run()
    assert set(path[:n]) == {-1} and count[0] == 0 and behind[0] == -1 and st == L.ST_BADDATA
    assert path[n:] == [0, 1] and count[1] == 2
    d.rows, d.off = [1024], torch.tensor([0, 1024])                    # the most there may be
    for name in ("parent", "token"):
        setattr(d, name, getattr(d, name)[:1024])
    d.target, d.draft, d.u_node, d.u_pick = d.target[:1024], d.draft[:1024], d.u_node[:1024], d.u_pick[:1]
    d.check()
    d.off, d.parent[5] = torch.tensor([5, 1024]), -1                   # rows 0 .. 4 are of no request
    path, count, behind, st = d.run()
    assert path[:7] == [55] * 5 + [0, 1] and count == [2] and st == 0   # (node 1 is a child of node 0: accepted)
    d.off = torch.tensor([0, 1025])
    path, count, behind, st = d.run()
    assert path == [55] * 1024 and count == [0] and behind == [-1] and st == L.ST_BADDATA


def test_chains_of_a_thousand():
    d = Drafts([1024], 17, seed=3)
    d.parent = list(range(-1, 1023))
    d.draft = d.target.clone()
    assert d.check() == [1024]
    g = Drafts([1024], 17, mode="greedy", seed=3)
    g.parent = list(range(-1, 1023))
    best = g.target.argmax(-1).tolist()
    g.token = [0] + best[:-1]
    assert g.check() == [1024]


def test_what_is_drawn_follows_the_target():
    # one draft, many uniform numbers: how often each token comes first is p, whatever q is
    V, N = 8, 40000
    g = torch.Generator().manual_seed(1)
    p, q = torch.softmax(torch.randn(V, generator=g), -1), torch.softmax(2 * torch.randn(V, generator=g), -1)
    d = Drafts([1], V, seed=0)
    B = 2000
    hits = torch.zeros(V)
    for k in range(N // B):
        d.rows, d.off = [3] * B, torch.arange(B + 1) * 3
        d.parent, d.token = [-1, 0, 0] * B, []
        draws = torch.multinomial(q, 2 * B, replacement=True, generator=g).tolist()
        for b in range(B):
            d.token += [0, draws[2 * b], draws[2 * b + 1]]
        d.target, d.draft = p.repeat(3 * B, 1), q.repeat(3 * B, 1)
        d.u_node, d.u_pick = torch.rand(3 * B, generator=g), torch.rand(B, generator=g)
        path, count, behind, st = d.run()
        for b in range(B):
            hits[d.token[3 * b + path[3 * b + 1]] if count[b] > 1 else behind[b]] += 1
    # a count of N p(1 - p) variance is within five standard deviations but once in a million
    assert ((hits - N * p).abs() <= 5 * (N * p * (1 - p)).sqrt()).all()


def test_another_stream_and_a_replayed_graph():
    L, dev = _lib(), "cuda"
    d = Drafts([6, 9], 5000, 3, seed=21)
    want = d.expected()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    path, count, behind, st = d.run(stream=s)
    assert (path, count, behind) == want
    i32 = dict(dtype=torch.int32, device=dev)
    args = [d.off.to(dev), torch.tensor(d.parent, **i32), torch.tensor(d.token, **i32), d.target.to(dev), torch.zeros(15, **i32),
            torch.zeros(2, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32)]
    kw = dict(draft=d.draft.to(dev), u_node=d.u_node.to(dev), u_pick=d.u_pick.to(dev))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        L.draft_verify(*args, **kw)
        with torch.cuda.graph(graph, stream=s):
            L.draft_verify(*args, **kw)
    for k in range(3):
        args[4].zero_()
        kw["u_node"].copy_(d.u_node)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert (args[4].tolist(), args[5].tolist(), args[6].tolist()) == d.expected()
        d.u_node = torch.rand(15, generator=torch.Generator().manual_seed(k))


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rows,vocab", [([128, 129, 1, 0, 127], 501), ([40, 3, 9], 20001), ([6] * 70, 4099), ([5] * 20, 33001),
                                        ([2] * 170, 3001), ([17], 60000)])
def test_greedy_with_few_and_many_nodes(rows, vocab, half):
    # requests whose rows are looked through at once stand beside those that are walked row by row
    t = Drafts(rows, vocab, reach=3, half=half, mode="greedy", seed=sum(rows))
    t.check()


@pytest.mark.parametrize("vocab", [300, 90001])
def test_greedy_nan_counts_where_the_walk_goes(vocab):
    # nodes 0 -> 1 -> 3 accepted, 2 not: only a NaN in a row of the path is reported, and no NaN is the largest
    t = Drafts([4, 4], vocab, mode="greedy", seed=9)
    t.parent = [-1, 0, 0, 1] * 2
    best = [int(r.argmax()) for r in t.target]
    t.token = [0, best[0], (best[0] + 1) % vocab, best[1], 0, best[4], (best[4] + 1) % vocab, best[5]]
    t.target[2, 7] = t.target[6, 250] = float("nan")
    assert t.check() == [3, 3]
    t.target[3, (best[3] + 5) % vocab] = float("nan")
    t.check(status=_lib().ST_NAN)
