"""echo_mla_tree over long contexts: pieces of several legs, whole ones and ones that are joined, longer than a wait may last."""
import math

import pytest
import torch

from _paged import EXP, SCORE, lse_tolerance, out_tolerance
from _speculate import TreeBatch, ancestors, random_parents

pytestmark = pytest.mark.gpu


def _lib():
    from sparse_attention_kv_echo_gb300 import lib
    return lib


@pytest.fixture
def short_waits():
    # a step of the kernel takes 1 to 4 us; the pieces of these tests take 600 us and more
    _lib().debug_wait_limit(200_000)
    yield
    _lib().debug_wait_limit(-1)


def _shared_pages(n, rows, heads, page, reach, seed):
    """One request of n tokens, `rows` of them its tree; a few pages hold all of them over and over."""
    g = torch.Generator().manual_seed(seed + 1)
    bt = TreeBatch([page], [1], [[{0}]], heads=heads, page=page, seed=seed, room=0)
    bt.lens, bt.rows, bt.n = [n], [rows], rows
    bt.seen = [ancestors(random_parents(rows, g, reach))]
    bt.q = torch.randn((rows, heads, 576), generator=g).to(torch.bfloat16)
    bt.tok_off, bt.tok_end, bt.row_off = torch.tensor([0, n]), torch.tensor([n]), torch.tensor([0, rows])
    bt.n_tokens, bt.tab = n, torch.zeros(-(-n // page), dtype=torch.int32)
    return bt


def _attend(bt):
    L, dev = _lib(), "cuda"
    row_off, q, tok_off, end, pages = bt.on(dev, L)
    words = -(-bt.n // 32)
    out = torch.full((bt.n, bt.heads, 512), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((bt.n, bt.heads), 7.0, device=dev)
    ws = torch.full((L.mla_chunk_workspace_size(bt.n, bt.heads, 1),), 0xFF, dtype=torch.uint8, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    L.mla_tree(row_off, q, bt.mask(words).to(dev), tok_off, bt.n_tokens, pages, bt.scale, out, lse, ws, st, tok_end=end)
    assert int(st) == 0
    return out.cpu(), lse.cpu()


def _expected(bt, i):
    """lse, out, sum w |v| and scale * max sum |q k| of row i: each cache row as often as the row sees it."""
    t = bt.visible(0, i)
    times = torch.bincount(bt.cache_row(0, t), minlength=bt.kv.shape[0]).double()
    kv, q = bt.kv.double(), bt.q[i].double()
    s = bt.scale * q @ kv.T + times.log()
    s = torch.where(times > 0, s, -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse[:, None])
    dots = bt.scale * (q.abs() @ kv[times > 0].abs().T).amax(-1)
    return lse, w @ kv[:, :512], w @ kv[:, :512].abs(), dots


@pytest.mark.parametrize("heads,kind", [(128, "rising"), (128, "falling"), (128, "empty"), (40, "rising"), (128, "nan")])
def test_pieces_of_several_legs(heads, kind, short_waits):
    # 100000 tokens a row, more groups of rows than clusters
    page, n, rows = 512, 100_000, 160 * (128 // heads)
    bt = _shared_pages(n, rows, heads, page, 7, 11)
    g = torch.Generator().manual_seed(4)
    pages = -(-n // page)
    bt.kv = torch.randn((4 * page, 576), generator=g).to(torch.bfloat16)
    order = torch.arange(pages) * 4 // pages                  # page 0 first, page 3 last
    bt.tab = (order if kind != "falling" else 3 - order).to(torch.int32)
    for i in range(4):                                        # longer keys, larger maxima
        bt.kv[i * page:(i + 1) * page] *= 0.5 + 0.5 * i
    if kind == "empty":                                       # nothing to see in the first and third quarters
        bt.tab[(order == 0) | (order == 2)] = -1
    if kind == "nan":
        bt.q[5, 3, 9] = float("nan")
    out, lse = _attend(bt)
    again = _attend(bt)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16))
    assert torch.equal(lse.view(torch.int32), again[1].view(torch.int32))
    for i in sorted({0, 1, 5, rows // 3, rows // 2, rows - 2, rows - 1}):
        ref, want, absv, dots = _expected(bt, i)
        hurt = torch.isnan(ref)
        assert torch.equal(hurt, torch.isnan(lse[i])) and torch.all(torch.isnan(out[i][hurt]))
        ok = ~hurt
        assert torch.all((lse[i].double() - ref).abs()[ok] <= lse_tolerance(dots, ref, 0)[ok])
        # (the value sums' accumulation may cut 2^-11 off over the tokens of a leg)
        tol = out_tolerance(want, absv, dots, 0) + absv * 2.0 ** -11
        assert torch.all((out[i].double() - want).abs()[ok] <= tol[ok])


def test_values_of_one_sign_over_a_million_tokens():
    # as the causal call's: a leg's sum may be cut short by 2^-12 on the mean
    bt = _shared_pages(1 << 20, 100, 128, 4096, 5, 7)
    bt.kv[:, :512] = bt.kv[:, :512].abs()
    out, lse = _attend(bt)
    for i in (0, 50, 99):
        ref, want, absv, dots = _expected(bt, i)
        assert torch.all((lse[i].double() - ref).abs() <= SCORE * dots + EXP * (1 + ref.abs()))
        off = (out[i].double() - want) / absv
        assert abs(float(off.mean())) <= 2.0 ** -12
        assert torch.all(off.abs() <= 2.0 ** -8 + 2 * SCORE * dots[:, None] * 1.01 + 2.0 ** -8 + 2.0 ** -10)
