"""Sampling under limits from long vocabularies, whose many small weights add up:
tokens and probabilities against 64 bits.  A sum of kept weights is good to 2^-25
of itself, so a uniform number lies within that of its token's part of the kept
sum, and so does the share at which top_p cuts."""
import math

import numpy as np
import pytest
import torch

import rank_markov_draft_amd as rmd

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# the stated bound on a sum, and as much again for the weights' own 2^-48, the
# uniform number's and the limits' parts of a sum (2^-40) many times over
TOL = 2.0 ** -25 + 2.0 ** -38


@pytest.fixture(autouse=True)
def room(native):
    yield
    torch.cuda.empty_cache()


def _fp32(v):
    return np.float32(v).item()


def _two_values(V, top, w, u, k, p, m, token, prob, what):
    """A row of the weight 1 at `top` and w elsewhere."""
    n = k if 0 < k < V else V
    if w < m:
        n = 1
    total, slack = 1.0 + (n - 1) * w, 0
    if p < 1:
        n = max(1, 1 + math.ceil((p * total - 1.0) / w))
        slack = math.ceil(2 * TOL * total / w) + 1
        total = 1.0 + (n - 1) * w
    rank = token - (top < token)                  # of the others before it
    assert token == top or 0 <= rank < n - 1 + slack, f"{what}: token {token} of the first {n} is not kept"
    mine = 1.0 if token == top else w
    before = min(rank, n - 1) * w + (1.0 if top < token else 0.0)
    assert before / total - 2 * TOL <= u <= (before + mine) / total + 2 * TOL, \
        f"{what}: {token} holds [{before / total}, {(before + mine) / total}), u is {u}"
    # one rounding to fp32, the sum, and where top_p cuts it
    assert abs(prob - mine / total) <= (2.0 ** -24 + 2 * TOL) * mine / total, f"{what}: probability {prob}, want {mine / total}"


# one logit above all others, which together weigh a tenth of the row, or each
# of them about a third of V / 2^62, the unit in which V weights of one can be summed
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tail", ["a tenth", "below a unit"])
@pytest.mark.parametrize("V", [2 ** 18, 2 ** 18 + 1, 2 ** 20 + 7, 2 ** 22, 2 ** 24 + 5, 2 ** 27 - 3])
def test_small_weights_add_up(native, V, tail, dtype):
    x_tail = -math.log(9 * V) if tail == "a tenth" else -(62 - math.ceil(math.log2(V)) + 1.5) * math.log(2)
    _rows_of_two_values(V, x_tail, dtype, [V // 3, 0], [2.0 ** -25, 0.05, 0.7, 1 - 2.0 ** -21, 1 - 2.0 ** -24])


@pytest.mark.parametrize("V", [2 ** 30 - 5])
def test_small_weights_add_up_in_the_largest_vocabulary(native, V):
    _rows_of_two_values(V, -23.0, BF16, [V // 3], [0.02, 0.95, 1 - 2.0 ** -24], short=True)


def _rows_of_two_values(V, x_tail, dtype, tops, us, short=False):
    x_tail = torch.tensor(x_tail, dtype=dtype).item()
    w = math.exp(x_tail)
    x = torch.full((len(tops), len(us), V), x_tail, dtype=dtype, device="cuda")
    for b, t in enumerate(tops):
        x[b, :, t] = 0.0
    u = torch.tensor([us] * len(tops), dtype=F32)
    for k, p, m in ((0, 0.999999, 0.0), (V // 2, 0.97, w / 2), (0, 1.0, 0.0), (0, 1 - 2.0 ** -24, 0.0), (V - 1, 1.0, 0.0),
                    (0, 1.0, w / 2), (0, 1.0, 2 * w), (200000, 1.0, 0.0), (300, 0.9, 0.0))[:3 if short else None]:
        p, m = _fp32(p), _fp32(m)
        tokens, probs = rmd.sample_block_filtered(x, u.cuda(), 1.0, top_k=k, top_p=p, min_p=m)
        tokens, probs = tokens.cpu(), probs.cpu()
        for b, t in enumerate(tops):
            for j in range(len(us)):
                _two_values(V, t, w, u[b, j].item(), k, p, m, tokens[b, j].item(), probs[b, j].item(),
                            f"V {V} top {t} u {us[j]} k {k} p {p} m {m}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [262144, 262145, 300001, 700007])
def test_random_rows(native, V, dtype):
    """Rows with a few tokens that stand out from a flat or a faint rest, under
    every kind of limit."""
    g = torch.Generator().manual_seed(V)
    x = torch.randn(6, 2, V, generator=g)
    x[2:4] = 2 * x[2:4] - 13.0
    x[4:] = 0.5 * x[4:] - 27.0
    x.scatter_(2, torch.randint(0, V, (6, 2, 5), generator=g), torch.rand(6, 2, 5, generator=g))
    x = x.to(dtype)
    u = torch.rand(6, 2, generator=g)
    u[:, 1] = 1.0 - 2.0 ** -24
    dev = x.cuda()
    for k, p, m in ((0, 1.0, 0.0), (0, 0.9, 0.0), (0, 1 - 2.0 ** -20, 0.0), (70, 1.0, 0.0), (V // 3, 1.0, 0.0), (V // 2, 0.999, 0.0),
                    (0, 1.0, 1e-13), (0, 0.99, 0.01), (100000, 0.95, 1e-6), (1500, 0.9, 0.0)):
        p, m = _fp32(p), _fp32(m)
        tokens, probs = rmd.sample_block_filtered(dev, u.cuda(), 0.75, top_k=k, top_p=p, min_p=m)
        for b in range(6):
            for j in range(2):
                _row(x[b, j].double().numpy(), u[b, j].item(), 0.75, k, p, m, tokens[b, j].item(), probs[b, j].item(),
                     f"V {V} row {b},{j} k {k} p {p} m {m}")


def _row(x, u, T, k, p, m, token, prob, what):
    V = x.size
    w = np.exp((x - x.max()) / T)
    order = np.argsort(-x, kind="stable")
    kept = np.zeros(V, bool)
    kept[order[:k] if 0 < k < V else order] = True
    kept &= w >= m
    maybe = kept
    if p < 1:
        by = order[kept[order]]
        upto = np.cumsum(w[by])
        before = upto - w[by]
        kept, maybe = np.zeros(V, bool), np.zeros(V, bool)
        kept[by[before < p * upto[-1]]] = True
        maybe[by[before < (p + TOL) * upto[-1]]] = True
    assert maybe[token], f"{what}: token {token} is not kept"
    total = math.fsum(w[kept])
    before = math.fsum(w[:token][kept[:token]])
    assert before / total - 2 * TOL <= u <= (before + w[token]) / total + 2 * TOL, \
        f"{what}: {token} holds [{before / total}, {(before + w[token]) / total}), u is {u}"
    assert abs(prob - w[token] / total) <= (2.0 ** -24 + 2 * TOL) * w[token] / total, f"{what}: probability {prob}"


def test_a_limit_that_is_hardly_on_changes_nothing(native):
    """The same rows with top_p off and just below 1: a tail of a tenth is drawn
    from as often."""
    V, n = 2 ** 25, 64
    row = torch.full((V,), -19.625, dtype=BF16, device="cuda")
    row[V // 2] = 0.0
    u = ((torch.arange(n, dtype=F32) + 0.5) / n).view(1, n).cuda()
    x = row.expand(1, n, V)
    off, _ = rmd.sample_block_filtered(x, u, 1.0)
    on, _ = rmd.sample_block_filtered(x, u, 1.0, top_p=1 - 2.0 ** -24)
    w = math.exp(-19.625)
    total = 1.0 + (V - 1) * w
    assert int((off != V // 2).sum()) == int((on != V // 2).sum()) > 0
    # as far apart as the roundings of the sum, and what top_p leaves out
    assert int((off - on).abs().max()) <= (2 * TOL + 2.0 ** -24) * total / w + 2
