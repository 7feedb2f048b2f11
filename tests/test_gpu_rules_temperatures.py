"""Drafts under rules at the ends of the temperature's range: a masked token is
never drawn, a token above -inf always can be."""
import numpy as np
import pytest
import torch

import rank_markov_draft_amd as rmd
from tests import rules_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# (B, V): drafts of a few rows a workgroup, and drafts by row tiles
SIZES = [(3, 300), (2, 1024), (64, 97), (70, 300), (200, 65)]


def _weights(V, r, dtype, scale=0.2):
    g = torch.Generator(device="cuda").manual_seed(V)
    return tuple((torch.randn(V, r, device="cuda", generator=g) * scale).to(dtype) for _ in range(2))


def _masked(B, M, V, dtype, seed):
    g = np.random.default_rng(seed)
    allowed = g.random((B, M, V)) < 0.3
    allowed[:, :, V // 2] = True
    allowed[-1, -1] = False
    x = torch.from_numpy(g.standard_normal((B, M, V)).astype(np.float32) * 3).to(dtype).cuda()
    return x, allowed, torch.from_numpy(ref.pack_mask(allowed)).cuda()


@pytest.mark.parametrize("T", [float("inf"), 1e60, 1e39])
@pytest.mark.parametrize("ldt,wdt", [(F32, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("B,V", SIZES)
def test_infinite_temperature_keeps_the_mask(native, B, V, ldt, wdt, T):
    """Scores are then the noise alone: the tokens are those of equal logits
    at a temperature of one; a row without an allowed token gives -1."""
    M = 2
    x, allowed, mask = _masked(B, M, V, ldt, B + V)
    w1, w2 = _weights(V, 16, wdt)
    first = torch.arange(B, device="cuda") % V
    tok, rows = rmd.sample_block_tokens_processed(x, first, w1, w2, T, token_mask=mask, seed=3)
    got = tok.cpu().numpy()
    assert got[-1, -1] == -1
    at = np.ones((B, M), bool)
    at[-1, -1] = False
    b, k = np.nonzero(at)
    assert (got[b, k] >= 0).all() and allowed[b, k, got[b, k]].all()
    even, _ = rmd.sample_block_tokens_processed(torch.zeros_like(x), first, w1 * 0, w2 * 0, 1.0, token_mask=mask, seed=3)
    assert torch.equal(tok, even)
    # -inf among the logits is a mask too, beside one or in its place
    y = torch.where(torch.from_numpy(allowed).cuda(), x, torch.full_like(x, -float("inf")))
    for kw in (dict(), dict(token_mask=mask)):
        assert torch.equal(rmd.sample_block_tokens_processed(y, first, w1, w2, T, seed=3, **kw)[0], tok)


@pytest.mark.parametrize("T", [float("inf"), 0.7])
@pytest.mark.parametrize("B,V", SIZES)
def test_infinities_are_drawn_first(native, B, V, T):
    """The first infinity that is allowed, whatever the noise; a NaN before it."""
    M = 2
    for ldt, wdt in ((F32, F32), (BF16, BF16)):
        x, allowed, mask = _masked(B, M, V, ldt, B + V + 2)
        x[:, :, ::2], x[0, 0, 2 * (V // 3)] = float("inf"), float("nan")
        allowed[0, 0, 2 * (V // 3)] = True
        mask = torch.from_numpy(ref.pack_mask(allowed)).cuda()
        w = torch.zeros(V, 16, dtype=wdt, device="cuda")
        first = torch.zeros(B, dtype=torch.int64, device="cuda")
        got = rmd.sample_block_tokens_processed(x, first, w, w, T, token_mask=mask, seed=8)[0].cpu().numpy()
        want = np.where(allowed[:, :, ::2].any(-1), 2 * allowed[:, :, ::2].argmax(-1), -2)
        want[0, 0] = 2 * (V // 3)
        want[-1, -1] = -1
        assert np.array_equal(got[want != -2], want[want != -2])


@pytest.mark.parametrize("T", [0.0, 0.1, 0.7, 1.5])
@pytest.mark.parametrize("ldt,wdt", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("B,V", SIZES)
def test_the_types_lowest_value_can_be_drawn(native, B, V, ldt, wdt, T):
    """Rows whose allowed tokens all hold the type's lowest value (an upstream
    mask of that value): they are above -inf, so one of them is drawn, the
    first, as the noise is lost beside them; one that holds more is drawn
    before them."""
    M, low = 2, torch.finfo(ldt).min
    _, allowed, mask = _masked(B, M, V, ldt, B + V + 1)
    x = torch.full((B, M, V), low, device="cuda").to(ldt)
    x[0, 1, V // 2] = -4.0
    w = torch.zeros(V, 8, dtype=wdt, device="cuda")
    first = torch.zeros(B, dtype=torch.int64, device="cuda")
    tok, rows = rmd.sample_block_tokens_processed(x, first, w, w, T, token_mask=mask, seed=5)
    want = np.where(allowed.any(-1), allowed.argmax(-1), -1)
    want[0, 1] = V // 2
    assert np.array_equal(tok.cpu().numpy(), want)
    assert torch.equal(rows > -float("inf"), torch.from_numpy(allowed).cuda())
