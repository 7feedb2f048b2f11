"""Sampling under limits: weights of tokens right beside a limit."""
import numpy as np
import pytest
import torch

import rank_markov_draft_amd as rmd

pytestmark = pytest.mark.gpu


def test_weights_next_to_min_p(native):
    """Tokens whose weight lies 2^-47 to 2^-43 of itself above or below min_p.
    A weight is off by 2^-50 for its polynomial, as much for its table, and |x|
    2^-52 for its exponent's roundings, 2^-48 in all for logits down to -7."""
    x = np.random.default_rng(15).uniform(-7.0, -0.25, 1 << 24).astype(np.float32)
    w = np.exp(x.astype(np.float64))                 # to 2^-52
    limit = w.astype(np.float32)
    apart = np.abs(w / limit.astype(np.float64) - 1.0)
    at = np.flatnonzero((apart >= 2.0 ** -47) & (apart <= 2.0 ** -43))
    assert at.size >= 32
    rows = torch.full((at.size, 1, 40), -float("inf"))
    rows[:, 0, 3] = 0.0
    rows[:, 0, 20] = torch.from_numpy(x[at])
    u = torch.full((at.size, 1), 1.0 - 2.0 ** -24)   # the second token wherever it is kept
    tokens, _ = rmd.sample_block_filtered(rows.cuda(), u.cuda(), 1.0, min_p=torch.from_numpy(limit[at]).cuda())
    want = np.where(w[at] >= limit[at].astype(np.float64), 20, 3)
    assert np.array_equal(tokens.view(-1).cpu().numpy(), want)
