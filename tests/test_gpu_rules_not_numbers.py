"""Infinities, NaN and the type's end values among the base logits of drafts
that run step by step, and in the greedy chain: masked and not, seen and not."""
import numpy as np
import pytest
import torch

import rank_markov_draft_amd as rmd
from tests import rules_reference as ref
from tests.test_gpu_logit_rules import _check_draft, _draft, _draft_case

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("T", [0.0, 0.7])
@pytest.mark.parametrize("B,V,ldt,wdt", [
    (4, 301, F32, F32), (4, 304, F32, BF16), (3, 1003, BF16, BF16), (6, 264, BF16, F32),   # a few rows a workgroup
    (70, 301, F32, F32), (66, 520, F32, BF16), (70, 131, BF16, BF16), (80, 136, BF16, F32),   # row tiles
    (6, 512, BF16, BF16), (64, 1024, BF16, BF16)])                                             # greedy: the chain
def test_logits_that_are_not_numbers(native, B, V, ldt, wdt, T):
    c = _draft_case(B, 3, V, 30, 12 if B % 2 else 16, ldt, wdt, mask="each", bias="row" if V % 2 else "shared")
    g = np.random.default_rng(B + V)
    # penalties whose products with the end values stay clear of the type's border
    c.rep = g.choice(np.array([1.5, 0.7, 2.0, 1.2], np.float32), B)
    low, top = torch.finfo(ldt).min, torch.finfo(ldt).max
    kinds = [[INF, -INF, NAN, low, top, 0.0, -0.0], [INF, -INF, low, top], [-INF, low], [-INF, top, 0.0], [-INF, NAN], [INF, 1.0],
             [-INF]]
    for b in range(B):
        for k in range(3):
            kind = kinds[(b * 3 + k) % len(kinds)]
            where = g.choice(V, V // 3, replace=False)
            if kind in ([-INF, low], [-INF]):
                where = np.arange(V)
            c.logits[b, k, torch.from_numpy(where)] = torch.tensor(g.choice(np.array(kind), len(where)), dtype=torch.float32).to(ldt)
    tok, rows = _draft(c, T, seed=21)
    masked = ~np.broadcast_to(c.allowed, (B, 3, V))
    assert (rows.cpu()[torch.from_numpy(masked)] == -INF).all()
    got = tok.cpu().numpy()
    drawn = got >= 0
    b, k = np.nonzero(drawn)
    assert not masked[b, k, got[b, k]].any()
    # rows on whose own values the order decides alone: the first NaN, else the first of the greatest
    own = rows.float().cpu().numpy()
    for b in range(B):
        for k in range(3):
            row = own[b, k]
            if np.isnan(row).any():
                assert got[b, k] == np.isnan(row).argmax()
            elif not (row > -INF).any():
                assert got[b, k] == -1
            elif T == 0.0 or row.max() == INF:
                # at a temperature a finite value whose score overflows ties with an infinity: it may stand before it
                first = int((row == row.max()).argmax())
                with np.errstate(over="ignore"):
                    over = row * np.float32(1.4426950408889634 / T) if T else row
                assert got[b, k] == (int((over == np.inf).argmax()) if T else first)
    # each row and token against the definition, where no score overflows
    if T == 0.0:
        _check_draft(c, tok, rows, T, 21)
