"""Plain forms of the calls of speculative decoding, from their definitions: lists, and torch in float64 on the CPU."""
import torch

from _paged import Batch


# ---------------------------------------------------------------- trees
def ancestors(parent):
    """For the parents of one request's nodes (-1 or out of range: none): the set of each node's ancestors and itself."""
    sets = []
    for i, p in enumerate(parent):
        sets.append({i} | (sets[p] if 0 <= p < i else set()))
    return sets


def mask_words(sets, words):
    """[n, words] int32, bit j % 32 of word j / 32."""
    rows = []
    for s in sets:
        w = [0] * words
        for j in s:
            w[j // 32] |= 1 << (j % 32)
        rows.append([x - (1 << 32) if x >= 1 << 31 else x for x in w])
    return torch.tensor(rows, dtype=torch.int64).to(torch.int32).view(len(sets), words)


def random_parents(n, g, reach):
    return [-1 if i == 0 else i - 1 - int(torch.randint(0, min(reach, i), (1,), generator=g)) for i in range(n)]


class TreeBatch(Batch):
    """A Batch whose new rows are tree nodes; seen[b][i]: the nodes row i of request b may see (those behind i are not
    seen either way)."""

    def __init__(self, lens, rows, seen, **kw):
        super().__init__(lens, rows, **kw)
        self.seen = seen

    def visible(self, b, i, window=0, sinks=0, sel=None):
        n, m = self.lens[b], self.rows[b]
        if n < m:
            return torch.zeros(0, dtype=torch.int64)
        t = torch.tensor(list(range(n - m)) + [n - m + j for j in sorted(self.seen[b][i]) if j <= i], dtype=torch.int64)
        return t[self.cache_row(b, t) >= 0]

    def mask(self, words):
        return torch.cat([mask_words(s, words) if s else torch.zeros((0, words), dtype=torch.int32) for s in self.seen])


# ---------------------------------------------------------------- verification
def verify(parent, token, target, draft, u_node, u_pick):
    """One request: (path, the token behind it), child by child, the residual carried along.  target, draft [n,vocab]
    (draft None: certain drafts); u_node None: greedy, the target's first best."""
    n = len(parent)
    v, path = 0, [0]
    while True:
        row = target[v].double()
        kids = [i for i in range(v + 1, n) if parent[i] == v]
        went = None
        if u_node is None:
            row = torch.where(row.isnan(), -torch.inf, row)
            ok = ~target[v].isnan()
            best = int((ok & (row == row[ok].max())).nonzero()[0]) if ok.any() else 0
            went = next((i for i in kids if token[i] == best), None)
            behind = best
        else:
            left, total = row, 1.0
            for i in kids:
                x = token[i]
                if not 0 <= x < row.numel():
                    continue
                if draft is None:
                    d = torch.zeros_like(row)
                    d[x] = 1.0
                else:
                    d = draft[v].double()
                if u_node[i] * float(d[x]) * total < float(left[x]):
                    went = i
                    break
                then = (left - total * d).clamp_min(0)
                if float(then.sum()) > 0:
                    left, total = then, float(then.sum())
            if went is None:
                c = left.cumsum(0)
                over = (c > u_pick * float(c[-1])).nonzero()
                behind = int(over[0]) if float(c[-1]) > 0 else 0
        if went is None:
            return path, behind
        v = went
        path.append(v)


# ---------------------------------------------------------------- pages
class Pool:
    """The pages' calls on lists.  kv: [layers, n_pages * page, ...]; bad / full: conditions seen."""

    def __init__(self, entries, n_pages, page, kv):
        self.tab, self.refs, self.page, self.kv = [-1] * entries, [0] * n_pages, page, kv
        self.bad = self.full = False

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def _consistent(self, off, end, b, tokens):
        lo, hi, e = off[b], off[b + 1], end[b]
        ok = 0 <= lo <= e <= hi <= tokens and lo % self.page == 0
        self.bad |= not ok
        return ok

    def _drop(self, p):
        if not 0 <= p < len(self.refs) or self.refs[p] <= 0:
            self.bad = True
        else:
            self.refs[p] -= 1

    def _copy(self, src, dst, rows):
        P = self.page
        self.kv[:, dst * P:dst * P + rows] = self.kv[:, src * P:src * P + rows].clone()

    def free(self, off, end, tokens):
        for b in range(len(end)):
            if not self._consistent(off, end, b, tokens):
                continue
            for e in range(-(-end[b] // self.page), -(-off[b + 1] // self.page)):
                if self.tab[e] != -1:
                    self._drop(self.tab[e])
                    self.tab[e] = -1

    def reserve(self, off, end, want, tokens):
        P, room = self.page, list(end)
        spare, refs, gone, copies, out_of = self.free_pages(), list(self.refs), [], [], False
        for b in range(len(end)):
            if not self._consistent(off, end, b, tokens):
                continue
            if not end[b] <= want[b] <= off[b + 1]:
                self.bad = True
                continue
            need, bad = [], False
            if want[b] > end[b]:
                for e in range(end[b] // P, -(-want[b] // P)):
                    p = self.tab[e]
                    part = e == end[b] // P and end[b] % P > 0
                    if p < 0:
                        bad |= part
                        need.append((e, -1, 0))
                    elif p >= len(refs) or refs[p] < 1:
                        bad = True
                    elif refs[p] > 1:
                        need.append((e, p, end[b] % P if part else 0))
            if bad:
                self.bad = True
                continue
            if need and (out_of or len(need) > len(spare)):
                self.full = out_of = True
                continue
            for e, p, rows in need:
                new = spare.pop(0)
                self.tab[e], self.refs[new] = new, 1
                if p >= 0:
                    gone.append(p)
                    copies.append((p, new, rows))
            room[b] = want[b]
        for p, new, rows in copies:
            self._copy(p, new, rows)
        for p in gone:
            self._drop(p)
        return room

    def fork(self, src, dst, off, end, tokens):
        P, B = self.page, len(end)
        pairs = []
        for i, (s, d) in enumerate(zip(src, dst)):
            ok = 0 <= s < B and 0 <= d < B and d not in src and d not in dst[:i]
            if ok:
                n = end[s] - off[s]
                ok = (0 <= off[s] <= end[s] <= off[s + 1] <= tokens and off[s] % P == 0 and
                      0 <= off[d] <= off[d + 1] <= tokens and off[d] % P == 0 and off[d + 1] - off[d] >= n)
            if not ok:
                self.bad = True
                continue
            pairs.append((s, d, n))
        def page_of(s, k):
            p = self.tab[off[s] // P + k]
            self.bad |= p >= len(self.refs)
            return p if 0 <= p < len(self.refs) else -1
        for s, d, n in pairs:
            for e in range(n // P):
                if page_of(s, e) >= 0:
                    self.refs[page_of(s, e)] += 1
        for s, d, n in pairs:
            for e in range(off[d] // P, -(-off[d + 1] // P)):
                if self.tab[e] != -1:
                    self._drop(self.tab[e])
                k = e - off[d] // P
                self.tab[e] = page_of(s, k) if k < n // P else -1
        spare = self.free_pages()
        for s, d, n in pairs:
            end[d] = off[d] + n
            p = page_of(s, n // P) if n % P else -1
            if p >= 0:
                if spare:
                    new = spare.pop(0)
                    self.tab[off[d] // P + n // P], self.refs[new] = new, 1
                    self._copy(p, new, n % P)
                else:
                    self.full = True
                    end[d] -= n % P

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        U = len(live)
        place = dict(zip([p for p in live if p >= U], [p for p in range(U) if self.refs[p] <= 0]))
        for a, z in place.items():
            self._copy(a, z, self.page)
            self.refs[z], self.refs[a] = self.refs[a], 0
        for e, p in enumerate(self.tab):
            if p >= U:
                if p in place:
                    self.tab[e] = place[p]
                else:
                    self.bad = True
        return U

    def keep(self, row_off, path, count, off, end, tokens):
        P, new_end = self.page, list(end)
        for b in range(len(end)):
            n, c = row_off[b + 1] - row_off[b], count[b]
            if not self._consistent(off, end, b, tokens):
                continue
            base = end[b] - n
            p = path[row_off[b]:row_off[b] + max(c, 0)]
            ok = 0 <= c <= n <= end[b] - off[b] and all(0 <= x < n for x in p) and all(x < y for x, y in zip(p, p[1:]))
            rows = []
            if ok:
                for i, x in enumerate(p):
                    if x == i:
                        continue
                    s, d = self.tab[(base + x) // P], self.tab[(base + i) // P]
                    if min(s, d) < 0 or max(s, d) >= len(self.refs) or self.refs[d] != 1:
                        ok = False
                        break
                    rows.append((s * P + (base + x) % P, d * P + (base + i) % P))
            if not ok:
                self.bad = True
                continue
            for s, d in rows:
                self.kv[:, d] = self.kv[:, s].clone()
            new_end[b] = base + c
        return new_end
