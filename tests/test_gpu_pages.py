"""The page calls and echo_rows_keep against their plain forms on lists: tables, counts and rows have to be equal."""
import random

import pytest
import torch

from _speculate import Pool

pytestmark = pytest.mark.gpu


def _lib():
    from sparse_attention_kv_echo_gb300 import lib
    return lib


class Both:
    """A pool on the GPU and on lists, driven alike."""

    def __init__(self, regions, n_pages, page, layers=2, seed=0, tail=0):
        L, dev = _lib(), "cuda"
        g = torch.Generator().manual_seed(seed)
        self.off = [0]
        for r in regions:
            self.off.append(self.off[-1] + r)
        self.tokens, self.B, self.page = self.off[-1] + tail, len(regions), page
        entries = -(-self.tokens // page)
        self.kv = torch.randn((layers, n_pages * page, 576), generator=g).to(torch.bfloat16)
        self.plain = Pool(entries, n_pages, page, self.kv.clone())
        i32 = dict(dtype=torch.int32, device=dev)
        self.pool = L.PagePool(torch.full((entries,), -1, **i32), torch.zeros(n_pages, **i32),
                               self.kv.to(dev) if layers > 1 else self.kv[0].to(dev), page)
        self.end = list(self.off[:-1])
        self.ws = torch.full((L.pages_workspace_size(max(self.B, 64), n_pages),), 255, dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, **i32)

    def put(self, x, dtype=torch.int64):
        return torch.tensor(x, dtype=dtype, device="cuda")

    def same(self):
        L = _lib()
        assert self.pool.page_tab.tolist() == self.plain.tab
        assert self.pool.refs.tolist() == self.plain.refs
        assert torch.equal(self.pool.kv.cpu().view(self.plain.kv.shape).view(torch.int16), self.plain.kv.view(torch.int16))
        st = int(self.status)
        assert bool(st & L.ST_BADDATA) == self.plain.bad and bool(st & L.ST_FULL) == self.plain.full
        assert not st & ~(L.ST_BADDATA | L.ST_FULL)
        self.status.zero_()
        self.plain.bad = self.plain.full = False

    def reserve(self, want, end=None):
        L = _lib()
        end = self.end if end is None else end
        room = torch.full((self.B,), -7, dtype=torch.int64, device="cuda")
        L.pages_reserve(self.put(self.off), self.put(end), self.put(want), self.tokens, self.pool, room, self.ws, self.status)
        got = room.tolist()
        assert got == self.plain.reserve(self.off, end, want, self.tokens)
        self.same()
        return got

    def free(self, end=None):
        L = _lib()
        end = self.end if end is None else end
        L.pages_free(self.put(self.off), self.put(end), self.tokens, self.pool, self.status)
        self.plain.free(self.off, end, self.tokens)
        self.same()

    def fork(self, src, dst):
        L = _lib()
        end = self.put(self.end)
        L.pages_fork(self.put(src, torch.int32), self.put(dst, torch.int32), self.put(self.off), end, self.tokens, self.pool,
                     self.ws, self.status)
        self.plain.fork(src, dst, self.off, self.end, self.tokens)
        assert end.tolist() == self.end
        self.same()

    def compact(self):
        L = _lib()
        used = torch.full((1,), -7, dtype=torch.int32, device="cuda")
        L.pages_compact(self.tokens, self.pool, used, self.ws, self.status)
        assert int(used) == self.plain.compact()
        self.same()

    def keep(self, row_off, path, count):
        L = _lib()
        new_end = torch.full((self.B,), -7, dtype=torch.int64, device="cuda")
        L.rows_keep(self.put(row_off), self.put(path, torch.int32), self.put(count, torch.int32), self.put(self.off),
                    self.put(self.end), self.tokens, self.pool, new_end, self.status)
        want = self.plain.keep(row_off, path, count, self.off, self.end, self.tokens)
        assert new_end.tolist() == want
        self.same()
        return want

    def fill(self, lengths):
        want = [self.off[b] + n for b, n in enumerate(lengths)]
        self.end = self.reserve(want)


@pytest.mark.parametrize("page,layers", [(1, 1), (16, 3), (7, 2), (64, 1)])
def test_requests_come_grow_and_go(page, layers):
    B = Both([40 * page, 0, 13 * page, 64 * page], 100, page, layers)
    B.fill([3 * page + 1, 0, 1, 40 * page])
    B.reserve([B.off[0] + 20 * page, B.off[1], B.off[2] + 13 * page, B.end[3]])
    B.free()                                                          # what was reserved goes again
    B.end = B.reserve([B.end[0] + 1, B.off[1], B.end[2] + 5, B.off[4]])
    B.end[3] = B.off[3]
    B.free()
    B.compact()
    B.fill([B.end[0] - B.off[0], 0, 13 * page, 50 * page])
    B.free(B.off[:-1])
    assert B.plain.tab == [-1] * len(B.plain.tab) and not any(B.plain.refs)
    B.compact()


def test_a_full_pool_serves_whole_requests_in_order():
    B = Both([160] * 5, 20, 16)
    assert B.reserve([160, 160 + 160, 320 + 16, 480, 640]) == [160, 320, 320, 480, 640]
    B.end = [160, 320, 320, 480, 640]
    B.free([100, 250, 320, 480, 640])
    B.end = [100, 250, 320, 480, 640]
    # seven pages are left: request 2 does not fit and takes nothing; 3 would, but comes behind; 0 needs none
    assert B.reserve([100, 250, 320 + 160, 480 + 16, 640]) == [100, 250, 320, 480, 640]
    assert B.reserve([112, 250, 320, 480 + 97, 640]) == [112, 250, 320, 577, 640]


def test_pages_that_others_hold_are_copied_on_write():
    page = 16
    B = Both([160] * 4, 40, page, layers=3)
    B.fill([50, 0, 0, 20])
    B.fork([0, 3, 3], [1, 2, 2])                                      # the third has a dst that is taken
    # two requests end within a page they share, both grow: both get a copy, the page has no holder left
    B.end[0], B.end[1] = B.off[0] + 40, B.off[1] + 40
    B.free()
    assert B.plain.refs[B.plain.tab[2]] == 2
    got = B.reserve([B.off[0] + 60, B.off[1] + 41, B.end[2], B.end[3]])
    assert got[0] == 60 and B.plain.tab[2] != B.plain.tab[B.off[1] // page + 2]
    # shared pages behind the end are replaced, not copied
    B.end = [B.off[0] + 16, B.off[1] + 41, B.end[2], B.end[3]]
    B.reserve([B.off[0] + 40, B.off[1] + 41, B.end[2], B.end[3]])


def test_forks():
    page = 16
    B = Both([128] * 9, 100, page)
    B.fill([100, 64, 5, 0, 30, 0, 0, 0, 0])
    B.fork([0, 0, 1, 2, 3], [5, 6, 7, 8, 4])                          # a full last page, one page, an empty context onto 4's
    B.fork([0], [4])
    B.fork([5, 5], [0, 1])                                            # the copies' copies; 0 and 1 give theirs up
    B.compact()
    B.fork([], [])


def test_pairs_that_cannot_be_forked_are_left_out():
    B = Both([64, 64, 32, 64, 64], 40, 16)
    B.fill([60, 20, 30, 0, 0])
    B.fork([0, 1, 3, -1, 0, 9, 0], [0, 4, 4, 3, 2, 3, 5])             # itself, fine, taken, no src, too short, no src, no dst
    B.fork([0, 1], [1, 3])                                            # 1 is a src: not overwritten


def test_a_fork_without_a_page_for_its_last_rows_ends_with_its_full_pages():
    B = Both([64] * 4, 6, 16)
    B.fill([60, 0, 0, 0])
    B.fork([0, 0, 0], [1, 2, 3])                                      # two pages are left for three tails
    assert B.end == [60, 64 + 60, 128 + 60, 192 + 48]


def test_compact_moves_what_lies_behind_the_used_places():
    for seed in range(4):
        rng = random.Random(seed)
        B = Both([160] * 12, 200, 16, layers=1 + seed % 2, seed=seed)
        B.fill([rng.randint(0, 160) for _ in range(12)])
        for b in rng.sample(range(12), 6):
            B.end[b] = rng.randint(B.off[b], B.end[b])
        B.free()
        B.compact()
        B.compact()                                                   # nothing to move


def test_compact_of_a_pool_of_many_pages():
    B = Both([50000] * 3, 130000, 1, layers=1)
    B.fill([50000, 30001, 12345])
    B.end[0] = 17
    B.free()
    B.compact()
    B.fill([20000, 30001, 50000])


def test_accepted_paths():
    page = 16
    B = Both([160] * 5, 60, page, layers=4)
    B.fill([100, 33, 16, 9, 3])
    row_off = [0, 12, 13, 29, 29, 32]
    path = [0, 2, 3, 7, 11] + [-1] * 7 + [0] + list(range(16)) + [0, 1, -1]
    B.end = B.keep(row_off, path, [5, 1, 16, 0, 2])
    assert B.end == [100 - 7, 160 + 33, 320 + 16, 480 + 9, 640 + 2]
    B.free()
    B.fill([n - o for n, o in zip([e + 3 for e in B.end], B.off)])


def test_paths_that_fit_no_tree_leave_the_request_as_it_was():
    page = 16
    B = Both([64] * 7, 60, page)
    B.fill([20, 20, 20, 20, 20, 20, 3])
    row_off = [0, 4, 8, 12, 16, 20, 24, 28]
    path = [0, 2, 2, -1] + [0, 3, 1, -1] + [0, 4, -1, -1] + [0, -1, 2, 3] + [0, 2, 3, -1] + [1, 3, -1, -1] + [0, 1, 2, -1]
    end = list(B.end)
    got = B.keep(row_off, path, [3, 3, 2, 3, 5, 2, 3])                # only the sixth is a path
    assert got == end[:5] + [end[5] - 2] + end[6:]
    got = B.keep(row_off, path, [-1, 0, 0, 0, 3, 0, 0])               # no count; nothing kept; a path


def test_paths_over_pages_of_others_or_of_none():
    page = 16
    B = Both([64] * 3, 20, page)
    B.fill([40, 0, 20])
    B.fork([0], [1])                                                  # pages 0 and 1 of it are shared now
    B.keep([0, 12, 24, 24], [2, 3] + [-1] * 10 + [5, 11] + [-1] * 10, [2, 2, 0])
    B.plain.tab[2], B.plain.tab[5] = -1, -1
    B.pool.page_tab[2] = B.pool.page_tab[5] = -1
    B.plain.refs = [B.plain.tab.count(p) for p in range(20)]
    B.pool.refs.copy_(torch.tensor(B.plain.refs, dtype=torch.int32))
    B.keep([0, 4, 4, 4], [1, 2, -1, -1], [2, 0, 0])                   # the rows have no page


def test_long_paths():
    B = Both([1024], 70, 16, layers=2)
    B.fill([1000])
    rng = random.Random(3)
    path = sorted(rng.sample(range(700), 300))
    B.keep([0, 700], path + [-1] * 400, [300])


def test_regions_off_a_page_border_and_inconsistent_bounds():
    B = Both([40, 56, 32], 30, 16, tail=5)                            # the second starts at token 40
    B.reserve([30, 40, 100])
    B.off = [0, 48, 96, 128]
    B.end = [10, 60, 96]
    B.reserve([20, 70, 100])                                          # partly used pages that are not there
    B.end = [0, 48, 96]
    B.end = B.reserve([20, 70, 100])
    for off, end in (([0, 48, 20, 128], [0, 48, 20]), ([0, 48, 96, 1000], [0, 48, 96]), ([-16, 48, 96, 128], [0, 48, 96]),
                     ([0, 48, 96, 128], [70, 30, 96])):
        B.off = off
        B.free(end)
        B.reserve([e + 1 for e in end], end)
        B.keep([0, 0, 0, 0], [], [0, 0, 0])


def test_entries_that_name_no_page():
    B = Both([64, 64], 8, 16)
    B.fill([64, 20])
    for bad in (8, 1 << 30):
        B.pool.page_tab[5] = bad
        B.plain.tab[5] = bad
        B.reserve([B.end[0], B.off[1] + 30])
        B.compact()
        B.fork([1], [0])
        B.free(B.off[:-1])
        B.fill([64, 20])


@pytest.mark.parametrize("seed", range(8))
def test_any_order_of_calls(seed):
    rng = random.Random(seed)
    page, n = rng.choice((1, 4, 16, 5)), rng.randint(2, 40)
    regions = [rng.randint(0, 12) * page for _ in range(n)]
    B = Both(regions, rng.randint(5, 6 * n + 5), page, layers=rng.randint(1, 3), seed=seed)
    for _ in range(40):
        what = rng.choice(("grow", "grow", "shrink", "fork", "compact", "keep"))
        if what == "grow":
            B.end = B.reserve([rng.randint(e, min(o, e + 4 * page)) for e, o in zip(B.end, B.off[1:])])
        elif what == "shrink":
            B.end = [e if rng.random() < 0.6 else rng.randint(o, e) for e, o in zip(B.end, B.off)]
            if rng.random() < 0.7:
                B.free()
        elif what == "fork":
            m = rng.randint(1, 6)
            B.fork([rng.randrange(-1, n + 1) for _ in range(m)], [rng.randrange(n) for _ in range(m)])
        elif what == "compact":
            B.compact()
        else:
            rows = [min(e - o, rng.randint(0, 9)) for e, o in zip(B.end, B.off)]
            row_off, path, count = [0], [], []
            for r in rows:
                c = rng.randint(0, r)
                path += sorted(rng.sample(range(r), c)) + [-1] * (r - c)
                count.append(c)
                row_off.append(row_off[-1] + r)
            B.end = B.keep(row_off, path, count)


@pytest.mark.parametrize("requests", [1024, 1025, 4096])
def test_many_requests(requests):
    page = 4
    B = Both([16] * requests, requests * 2 + 9, page, layers=1)
    rng = random.Random(requests)
    B.fill([rng.randint(0, 6) for _ in range(requests)])
    B.end = B.reserve([min(e + rng.randint(0, 16), o) for e, o in zip(B.end, B.off[1:])])   # the pool runs out
    pairs = rng.sample(range(requests), 600)
    B.ws = torch.full((_lib().pages_workspace_size(requests, B.plain.refs.__len__()),), 255, dtype=torch.uint8, device="cuda")
    B.free()
    B.fork(pairs[:300], pairs[300:])
    B.compact()


def test_a_step_of_the_pages_in_a_replayed_graph():
    L, page = _lib(), 16
    B = Both([320] * 3, 80, page, layers=2)
    B.fill([100, 37, 200])
    row_off, path, count = [0, 6, 7, 12], [0, 2, 5, -1, -1, -1, 0, 0, 1, 4, -1, -1], [3, 1, 3]
    off, end, new_end, room = B.put(B.off), B.put(B.end), B.put([0] * 3), B.put([0] * 3)
    ro, pa, co, nodes = B.put(row_off), B.put(path, torch.int32), B.put(count, torch.int32), B.put([6, 1, 5])
    want = B.put([0] * 3)

    def step():
        L.rows_keep(ro, pa, co, off, end, B.tokens, B.pool, new_end, B.status)
        L.pages_free(off, new_end, B.tokens, B.pool, B.status)
        torch.add(new_end, nodes, out=want)
        L.pages_reserve(off, new_end, want, B.tokens, B.pool, room, B.ws, B.status)
        end.copy_(room)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        step()
    torch.cuda.synchronize()
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        mid = B.plain.keep(row_off, path, count, B.off, B.end, B.tokens)
        B.plain.free(B.off, mid, B.tokens)
        B.end = B.plain.reserve(B.off, mid, [m + n for m, n in zip(mid, [6, 1, 5])], B.tokens)
        assert end.tolist() == B.end
        B.same()
