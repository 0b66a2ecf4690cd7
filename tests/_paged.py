"""Plain 64-bit forms of the operators over a paged latent cache, and inputs for their tests.

Everything here is torch in float64 on the CPU, one row at a time, from the definitions."""
import math

import torch

DQK, DV = 576, 512


class Batch:
    """A batch of requests over a paged cache.  lens / rows: tokens and new rows per request."""

    def __init__(self, lens, rows, heads=128, page=64, seed=0, absent=0.0, room=3, lead=0, spare_pages=2, per_request=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.rows, self.heads, self.page = list(lens), list(rows), heads, page
        B = len(lens)
        regions = [n + room for n in lens]
        regions[0] += lead
        off = torch.tensor([0] + regions, dtype=torch.int64).cumsum(0)
        self.n_tokens = int(off[-1])
        self.tok_off = off
        self.tok_end = off[:-1] + torch.tensor(list(lens), dtype=torch.int64)
        self.row_off = torch.tensor([0] + list(rows), dtype=torch.int64).cumsum(0)
        self.n = int(self.row_off[-1])
        pages = -(-self.n_tokens // page)
        self.req_rows = per_request
        if per_request:                                  # each request's rows at random places of its own pool
            assert page == 1
            self.tab = torch.full((self.n_tokens,), -1, dtype=torch.int32)
            for b in range(B):
                r = torch.randperm(per_request, generator=g)[:regions[b]].to(torch.int32)
                self.tab[int(off[b]):int(off[b + 1])] = r
            kv_rows = B * per_request
        else:
            self.tab = torch.randperm(pages + spare_pages, generator=g)[:pages].to(torch.int32)
            kv_rows = (pages + spare_pages) * page
        if absent:
            self.tab[torch.rand(self.tab.numel(), generator=g) < absent] = -1
        self.kv = torch.randn((kv_rows, DQK), generator=g).to(torch.bfloat16)
        self.q = torch.randn((self.n, heads, DQK), generator=g).to(torch.bfloat16)
        self.scale = 1.0 / math.sqrt(192.0)

    def cache_row(self, b, t):
        """Cache row of each token of t (tensor), -1 where absent."""
        at = self.tok_off[b] + t
        e = self.tab[torch.div(at, self.page, rounding_mode="floor")].long()
        r = b * self.req_rows + e * self.page + at % self.page
        return torch.where(e < 0, torch.full_like(r, -1), r)

    def visible(self, b, i, window=0, sinks=0, sel=None):
        """Tokens row i of request b sees, with repetitions, those without a row left out."""
        n, p = self.lens[b], self.lens[b] - self.rows[b] + i
        if p < 0 or n < self.rows[b]:
            return torch.zeros(0, dtype=torch.int64)
        if sel is not None:
            t = sel[int(self.row_off[b]) + i].long()
            t = t[(t >= 0) & (t < n)]
        else:
            t = torch.arange(p + 1)
            if window:
                t = t[(t > p - window) | (t < sinks)]
        return t[self.cache_row(b, t) >= 0]

    def attend(self, window=0, sinks=0, sel=None):
        """out, lse, and the two scales of their errors: sum w |v| and scale * max_t sum_d |q_d k_d|."""
        H = self.heads
        out = torch.zeros((self.n, H, DV), dtype=torch.float64)
        lse = torch.full((self.n, H), -math.inf, dtype=torch.float64)
        absv = torch.zeros_like(out)
        dots = torch.zeros((self.n, H), dtype=torch.float64)
        kv = self.kv.double()
        for b in range(len(self.lens)):
            for i in range(self.rows[b]):
                r = int(self.row_off[b]) + i
                t = self.visible(b, i, window, sinks, sel)
                if t.numel() == 0:
                    continue
                k = kv[self.cache_row(b, t)]
                q = self.q[r].double()
                s = self.scale * q @ k.T
                lse[r] = torch.logsumexp(s, -1)
                w = torch.exp(s - lse[r][:, None])
                out[r] = w @ k[:, :DV]
                absv[r] = w @ k[:, :DV].abs()
                dots[r] = self.scale * (q.abs() @ k.abs().T).amax(-1)
        return out, lse, absv, dots

    def weigh(self, lse, mass, mass_out, decay, window=0, sinks=0):
        """mass_out and the error scale of each entry: sum over rows and heads of w * (scale * sum |q k|)."""
        new, err = mass_out.double().clone(), torch.zeros(self.n_tokens, dtype=torch.float64)
        kv = self.kv.double()
        for b in range(len(self.lens)):
            lo, hi = int(self.tok_off[b]), int(self.tok_end[b])
            new[lo:hi] = decay * mass[lo:hi].double() if decay else 0.0
            for i in range(self.rows[b]):
                r = int(self.row_off[b]) + i
                t = self.visible(b, i, window, sinks)
                if t.numel() == 0:
                    continue
                k, q = kv[self.cache_row(b, t)], self.q[r].double()
                ls = lse[r].double()
                w = torch.exp(self.scale * q @ k.T - ls[:, None])
                w[torch.isinf(ls)] = 0.0
                new[lo + t] += w.sum(0)
                err[lo + t] += (w * (self.scale * q.abs() @ k.abs().T + ls.abs()[:, None] + 1)).sum(0)
        return new, err

    def on(self, dev, lib):
        """The device tensors of a call: (row_off, q, tok_off, tok_end, pages)."""
        tab, kv = self.tab.to(dev), self.kv.to(dev)
        return (self.row_off.to(dev), self.q.to(dev), self.tok_off.to(dev), self.tok_end.to(dev),
                lib.KVPages(tab, kv, self.page, self.req_rows))


# A score is an fp32 sum of 576 exact products, in at most 36 steps of 16: at most 36 + 16 roundings of
# half a step (2^-24) each, taken twice for an accumulator that truncates: 104 * 2^-24 of sum |q k|, below 2^-17.
SCORE = 2.0 ** -17
# exp and log of a score in fp32: scaling and subtraction round |s| and |lse| by 2^-24 each, a base-2
# exponential is good to 2^-22, and a sum of n weights in any order is off by less than n * 2^-24.
EXP = 2.0 ** -20


def lse_tolerance(dots, lse, n):
    return SCORE * dots + EXP * (1 + lse.abs().nan_to_num(0.0, 0.0, 0.0)) + n * 2.0 ** -24


def out_tolerance(out, absv, dots, n):
    """The weights rounded to bf16 (half a step is 2^-8 of the value), the scores' errors (twice: in the weight and
    in the sum that divides it), and the result rounded to bf16."""
    rel = 2.0 ** -8 + 2 * (SCORE * dots[..., None] * 1.01 + 8 * EXP + n * 2.0 ** -24)
    return (rel * absv) * (1 + 2.0 ** -8) + 2.0 ** -8 * out.abs() + 1e-30


def victims(slot2tok, mass, off, length, keep, sinks, recent):
    """(tokens, slots) of the victims, by a plain sort, slots ascending."""
    held = [(s, int(t)) for s, t in enumerate(slot2tok.tolist()) if 0 <= t < length]
    may = [(float(mass[off + t]) + 0.0, t, s) for s, t in held if sinks <= t < length - recent]
    want = max(0, min(len(held) - keep, len(may)))
    got = sorted((s, t) for _, t, s in sorted(may)[:want])
    return [t for _, t in got], [s for s, _ in got]
