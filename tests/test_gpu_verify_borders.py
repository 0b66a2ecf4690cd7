"""echo_draft_verify where a test or a draw falls next to its border: uniform numbers with bits below 2^-32, and
probabilities next to what earlier rejections took of them."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from _speculate import verify

pytestmark = pytest.mark.gpu


def _run(rows, parent, token, target, draft, u_node, u_pick):
    from sparse_attention_kv_echo_gb300 import lib as L
    dev, B, n = "cuda", len(rows), len(parent)
    i32 = dict(dtype=torch.int32, device=dev)
    off = torch.tensor([0] + rows, dtype=torch.int64).cumsum(0).to(dev)
    path, count, behind, status = (torch.zeros(k, **i32) for k in (n, B, B, 1))
    L.draft_verify(off, torch.tensor(parent, **i32), torch.tensor(token, **i32), target.to(dev), path, count, behind, status,
                   draft=None if draft is None else draft.to(dev), u_node=torch.tensor(u_node, device=dev),
                   u_pick=torch.tensor(u_pick, device=dev))
    assert int(status) == 0
    path, at, got = path.tolist(), 0, []
    for m, c, y in zip(rows, count.tolist(), behind.tolist()):
        got.append((path[at:at + c], y))
        at += m
    return got


def _want(rows, parent, token, target, draft, u_node, u_pick):
    at, want = 0, []
    for b, m in enumerate(rows):
        s = slice(at, at + m)
        want.append(verify(parent[s], token[s], target[s], None if draft is None else draft[s], u_node[s], u_pick[b]))
        at += m
    return want


def _f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


# The tests below are 2^-49 and more off their borders: u is a multiple of 2^-64 and enters whole, and a product u d R is
# cut off below 2^-57 (R, where it is not 1, is a sum of four values, good to 2^-43; u d is below 2^-14 there, and the
# margin 2^-36).
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("low,high", [(-39, -32), (-33, -24), (-25, -8)])
def test_a_draft_of_small_probability(low, high, half):
    # certain drafts: accepted below p, whatever bits u has
    g = torch.Generator().manual_seed(-low)
    B, dtype = 200, torch.bfloat16 if half else torch.float32
    p = (2.0 ** (low + (high - low) * torch.rand(B, generator=g))).to(dtype)
    target = torch.zeros((2 * B, 4), dtype=dtype)
    target[0::2, 1], target[0::2, 3], target[1::2, 2] = p, 1.0, 1.0
    u = [0.5, 0.0] * B
    for b in range(B):
        u[2 * b + 1] = _f32(float(p[b]) * (1 + (1 if b % 2 else -1) * 2.0 ** -10))
    args = [2] * B, [-1, 0] * B, [0, 1] * B, target, None, u, [0.5] * B
    got = _run(*args)
    assert got == _want(*args)
    assert [len(x[0]) for x in got] == [1 if b % 2 else 2 for b in range(B)]


def test_a_second_child_against_what_little_is_left():
    # node 1's token has no probability; node 2's left is p - d, some 2^-24 where d is a half, R the sum of what is left
    g = torch.Generator().manual_seed(5)
    B, V = 200, 4
    target, draft = torch.zeros((3 * B, V)), torch.zeros((3 * B, V))
    u = [0.5, 0.9, 0.0] * B
    for b in range(B):
        k = int(torch.randint(1, 60, (1,), generator=g))
        draft[3 * b] = torch.tensor([0.25, 0.5, 0.0, 0.125])
        target[3 * b] = torch.tensor([0.0, 0.5 + k * 2.0 ** -24 * 2, 0.25, 0.125])
        left = (target[3 * b].double() - draft[3 * b].double()).clamp_min(0)
        border = float(left[1]) / (0.5 * float(left.sum()))
        u[3 * b + 2] = _f32(border * (1 + (1 if b % 2 else -1) * 2.0 ** -13))
        target[3 * b + 2, 3] = 1.0
    args = [3] * B, [-1, 0, 0] * B, [0, 0, 1] * B, target, draft, u, [0.5] * B
    got = _run(*args)
    assert got == _want(*args)
    assert [len(x[0]) for x in got] == [1 if b % 2 else 2 for b in range(B)]


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("low,high", [(-39, -32), (-33, -24), (-25, -8)])
def test_a_token_of_small_probability_in_front(low, high, half):
    # the first token is drawn below p / (p + 1): a sum of two values, exact to 2^-60
    g = torch.Generator().manual_seed(-high)
    B, dtype = 200, torch.bfloat16 if half else torch.float32
    p = (2.0 ** (low + (high - low) * torch.rand(B, generator=g))).to(dtype)
    target = torch.zeros((B, 40), dtype=dtype)
    target[:, 0], target[:, 37] = p, 1.0
    pick = [_f32(float(p[b]) / (1 + float(p[b])) * (1 + (1 if b % 2 else -1) * 2.0 ** -10)) for b in range(B)]
    args = [1] * B, [-1] * B, [0] * B, target, None, [0.5] * B, pick
    got = _run(*args)
    assert got == _want(*args)
    assert [y for _, y in got] == [37 if b % 2 else 0 for b in range(B)]


# ---------------------------------------------------------------- what is left of p next to S d
def _floor32(x):
    """The largest float32 at or below the fraction x > 0."""
    f = np.float32(float(x))
    return f if Fraction(float(f)) <= x else np.nextafter(f, np.float32(0))


def _knife(scales, steps, seed):
    """A node's p and d (float32 rows) whose first two rejections (of tokens 0 and 1, without probability) leave S =
    1 + 2^-8 - 0.49 * 2^-23: its upper 24 bits round S up, so that S d lies below the product of those, by nearly an ulp where
    d is close under a power of two.  One token for each of scales: d about that much, p the float next to S d but `steps` of
    them; four more tokens bring the sum of max(0, p - d) to S - 1 and have nothing left at S.
    Returns p, d and the exact rest of every token at S."""
    rng = np.random.default_rng(seed)
    upper = np.float32(1 + 2.0 ** -8)
    want = Fraction(float(upper)) - Fraction(49, 100) * Fraction(1, 2 ** 23)
    p, d = [np.float32(0)] * 2, [np.float32(2.0 ** -10)] * 2
    for scale, step in zip(scales, steps):
        while True:
            dy = np.float32(scale * (0.98 + 0.01 * rng.random()))
            x = upper * dy                                             # rounded to float32
            py = x
            for _ in range(abs(step)):
                py = np.nextafter(py, np.float32(step))
            rest = Fraction(float(py)) - want * Fraction(float(dy))
            if step >= 0 or rest > Fraction(float(np.spacing(x))) / 8:  # below x, and something left all the same
                break
        p.append(py)
        d.append(dy)
    lack = want - 1 - sum(Fraction(float(a)) - Fraction(float(b)) for a, b in zip(p[2:], d[2:]))
    sizes = [Fraction(3, 4), Fraction(1, 2 ** 14), Fraction(1, 2 ** 26), Fraction(1, 2 ** 38), Fraction(0)]
    for size, smaller in zip(sizes, sizes[1:]):
        pz = _floor32(size + lack - (want - 1) * smaller / 2)
        assert size < Fraction(float(pz)) < want * size
        lack -= Fraction(float(pz)) - size
        p.append(pz)
        d.append(np.float32(float(size)))
    p, d = np.array(p), np.array(d)
    S = 1 + sum(max(Fraction(0), Fraction(float(a)) - Fraction(float(b))) for a, b in zip(p, d))
    assert abs(S - want) < Fraction(1, 2 ** 49) and p.sum() < 8 and d.sum() < 8
    return p, d, [max(Fraction(0), Fraction(float(a)) - S * Fraction(float(b))) for a, b in zip(p, d)]


@pytest.mark.parametrize("scales,steps", [([0.5], [-1]), ([0.25, 0.5], [-1, -1]), ([0.5, 0.25, 0.125, 0.0625], [-1, 0, 1, -1]),
                                          ([0.0625] * 10, [-1] * 10), ([0.25, 0.125, 0.125, 0.25], [1, 2, -1, 0])])
@pytest.mark.parametrize("seed", range(3))
def test_a_rest_below_the_last_place(scales, steps, seed):
    # what is left is some 2^-25 to 2^-29 of each token, good to 2^-45: draws in the middle of each one's share, and, of a
    # third child, tests a 64th above and below the border
    p, d, rest = _knife(scales, steps, seed)
    total, V = sum(rest), len(p)
    row, drawn = torch.from_numpy(p), torch.from_numpy(d)
    rows, parent, token, u, pick, want = [], [], [], [], [], []
    run = Fraction(0)
    for y in range(V):
        if rest[y] > total / 1000:
            rows.append(3)
            parent += [-1, 0, 0]
            token += [0, 0, 1]
            u += [0.5, 0.5, 0.5]
            pick.append(float((run + rest[y] / 2) / total))
            want.append(([0], y))
            border = rest[y] / (Fraction(float(d[y])) * total)
            if border < Fraction(63, 64):
                for side in (-1, 1):
                    rows.append(4)
                    parent += [-1, 0, 0, 0]
                    token += [0, 0, 1, y]
                    u += [0.5, 0.5, 0.5, float(border * (1 + Fraction(side, 64)))]
                    pick.append(0.0)
                    want.append(([0, 3], 0) if side < 0 else None)     # (a third rejection leaves other tokens)
        run += rest[y]
    assert want
    n = len(parent)
    target, draft = torch.zeros((n, V)), torch.zeros((n, V))
    at = 0
    for m in rows:
        target[at], draft[at] = row, drawn
        if m == 4:
            target[at + 3, 0] = 1.0
        at += m
    got = _run(rows, parent, token, target, draft, u, pick)
    for g, w in zip(got, want):
        assert g == w if w else g[0] == [0]
