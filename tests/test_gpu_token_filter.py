"""Sampling under temperature, top-k, top-p and min-p on the GPU against 64
bits: tokens equal, probabilities to their last rounding."""
import math

import numpy as np
import pytest
import torch

import rank_markov_draft_amd as rmd
from tests import filter_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def _check(x, u, T, k, p, m, tokens, probs, what):
    """Every row; T, k, p, m are lists by request."""
    B, M, V = x.shape
    X, tokens, probs = x.double().numpy(), tokens.cpu(), probs.cpu()
    for b in range(B):
        for j in range(M):
            args = (u[b, j].item(), T[b], k[b], p[b], m[b])
            want, prob, near = ref.row(X[b, j], *args)
            got = tokens[b, j].item()
            # A border closer than this (2^-39.8 of the sum) may fall to either
            # side: each weight is good to 2^-42 of itself, a sum of them and its
            # part by top_p or u with it, a sum's roundings to 2^-45
            if near > 1e-12:
                assert got == want, f"{what} row {b},{j} {args}: {got}, want {want}"
                if math.isnan(prob):
                    assert math.isnan(probs[b, j].item())
                else:
                    # one rounding to fp32, and the weights' 2^-40
                    assert abs(probs[b, j].item() - prob) <= (2.0 ** -24 + 2.0 ** -38) * prob + 2.0 ** -149, f"{what} row {b},{j} {args}"
            else:
                assert what.startswith("borders"), f"{what} row {b},{j}: no border this close is meant"


def _limits(B, kind, g):
    T = (0.4 + torch.rand(B, generator=g)).tolist()
    k, p, m = [0] * B, [1.0] * B, [0.0] * B
    T = [np.float32(t).item() for t in T]
    for b in range(B):
        one = kind if kind != "mixed" else ["greedy", "none", "top_k", "top_p", "min_p", "all", "wide_k"][b % 7]
        if one == "greedy":
            T[b] = 0.0
        if one in ("top_k", "all"):
            k[b] = int(torch.randint(1, 90, (1,), generator=g))
        if one == "wide_k":
            k[b] = int(torch.randint(400, 30000, (1,), generator=g))
        if one in ("top_p", "all"):
            p[b] = np.float32(0.05 + 0.949 * torch.rand(1, generator=g).item()).item()
        if one in ("min_p", "all"):
            m[b] = np.float32(0.3 * torch.rand(1, generator=g).item() ** 2).item()
    return T, k, p, m


def _call(x, u, T, k, p, m, **kw):
    dev = dict(temperature=torch.tensor(T, dtype=F32).cuda(), top_k=torch.tensor(k).cuda(),
               top_p=torch.tensor(p, dtype=F32).cuda(), min_p=torch.tensor(m, dtype=F32).cuda())
    return rmd.sample_block_filtered(x.cuda(), u.cuda(), dev.pop("temperature"), **dev, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["none", "top_k", "top_p", "min_p", "all", "mixed", "wide_k"])
@pytest.mark.parametrize("B,M,V", [(1, 1, 1), (2, 1, 3), (3, 2, 130), (7, 2, 1000), (7, 1, 8192), (7, 2, 32003), (3, 1, 129280)])
def test_limits(native, B, M, V, kind, dtype):
    g = torch.Generator().manual_seed(B + M + V)
    x = 2 * torch.randn(B, M, V, generator=g)
    x.scatter_add_(2, torch.randint(0, V, (B, M, 20), generator=g), 10 * torch.rand(B, M, 20, generator=g))
    x = x.to(dtype)
    u = torch.rand(B, M, generator=g)
    lim = _limits(B, kind, g)
    tokens, probs = _call(x, u, *lim)
    assert tokens.dtype == torch.int64 and probs.dtype == F32 and tuple(tokens.shape) == (B, M) == tuple(probs.shape)
    _check(x, u, *lim, tokens, probs, f"{kind} V {V}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_flat_rows(native, dtype):
    """Rows in which tens of thousands of tokens are kept, whose borders lie
    among them."""
    g = torch.Generator().manual_seed(4)
    B, V = 9, 50257
    x = torch.randn(B, 1, V, generator=g).to(dtype)
    u = torch.rand(B, 1, generator=g)
    lim = ([1.0, 2.0, 1.0, 5.0, 1.0, 1.0, 1e9, 1.0, 0.3], [0, 0, 9000, 20000, 600, 513, 0, 45000, 512],
           [0.5, 0.9, 1.0, 0.7, 0.25, 1.0, 0.4, 0.999, 0.97], [0.0, 0.0, 0.0, 0.0, 0.01, 0.05, 0.0, 0.0001, 0.0])
    lim = tuple([np.float32(v).item() if isinstance(v, float) else v for v in part] for part in lim)
    tokens, probs = _call(x, u, *lim)
    _check(x, u, *lim, tokens, probs, "flat")


@pytest.mark.parametrize("V", [5, 700, 2049, 30000])
def test_equal_logits(native, V):
    """Ties go to the lowest index; a border among thousands of equal tokens."""
    ks = [1, 3, V - 1, 0, 0, 0, V // 2, 0]
    ps = [1.0, 1.0, 1.0, 0.5, 0.25, 0.0, 0.5, 0.875]
    B = len(ks)
    x = torch.full((B, 2, V), -3.25)
    x[7, :, V // 2:] = -4.0
    g = torch.Generator().manual_seed(V)
    u = torch.rand(B, 2, generator=g)
    u[:, 1] = 1.0 - 2.0 ** -24
    lim = ([1.0] * B, ks, ps, [0.0] * B)
    tokens, probs = _call(x, u, *lim)
    for b in range(7):
        # weights of one: everything is exact, at the borders too
        n = min(ks[b], V) if ks[b] > 0 else V
        n = max(1, math.ceil(ps[b] * n)) if ps[b] < 1 else n
        for j in range(2):
            assert tokens[b, j].item() == int(u[b, j].double().item() * n), (b, j)
            assert probs[b, j].item() == np.float32(1.0 / n).item()
    _check(x[7:], u[7:], [1.0], [0], [0.875], [0.0], tokens[7:], probs[7:], "two values")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_ties(native, dtype):
    """A handful of values a thousandfold each, so that every border falls among equal tokens."""
    g = torch.Generator().manual_seed(6)
    B, V = 8, 40001
    x = (torch.randint(-8, 3, (B, 1, V), generator=g).float() * 0.5).to(dtype)
    u = torch.rand(B, 1, generator=g)
    lim = ([1.0] * B, [0, 5000, 0, 2000, 100, 0, 7, 39999], [0.9, 1.0, 0.33, 0.7, 1.0, 1.0, 0.5, 0.95],
           [0.0, 0.0, 0.0, 0.0, 0.0, 0.2, 0.0, 0.0])
    lim = tuple([np.float32(v).item() if isinstance(v, float) else v for v in part] for part in lim)
    tokens, probs = _call(x, u, *lim)
    _check(x, u, *lim, tokens, probs, "ties")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_numbers_of_candidates(native, dtype):
    """As many kept tokens as the ways of placing them hold, and one more or
    less; with top_p and min_p inside them, and -inf above the k-th."""
    g = torch.Generator().manual_seed(21)
    ks = [1, 2, 63, 64, 65, 127, 128, 129, 130, 500, 2047, 2048, 2049, 2050]
    V = 33001
    x = torch.randn(len(ks), 3, V, generator=g)
    x[:, 1] = torch.round(4 * x[:, 1]) / 4                       # ties at every border
    x[:, 2, torch.randperm(V, generator=g)[100:]] = -INF         # never more than 100
    x = x.to(dtype)
    u = torch.rand(len(ks), 3, generator=g)
    ones, zeros = [1.0] * len(ks), [0.0] * len(ks)
    for T, p, m in ((1.0, 1.0, 0.0), (0.5, 0.75, 0.0), (2.0, 1.0, 0.125), (1.0, 0.9375, 0.0625)):
        lim = ([T] * len(ks), ks, [p] * len(ks), [m] * len(ks))
        tokens, probs = _call(x, u, *lim)
        _check(x, u, *lim, tokens, probs, f"candidates T {T} p {p} m {m}")
    # the same number of tokens left by a mask of -inf, no limit on
    for b, k in enumerate(ks):
        x[b, 0, torch.randperm(V, generator=g)[k:]] = -INF
    tokens, probs = _call(x, u, ones, [0] * len(ks), ones, zeros)
    _check(x, u, ones, [0] * len(ks), ones, zeros, tokens, probs, "candidates masked")


def test_masks_and_special_rows(native):
    g = torch.Generator().manual_seed(7)
    B, V = 14, 9000
    x = 2 * torch.randn(B, 1, V, generator=g)
    x[0] = -INF                                       # nothing
    x[1] = -INF
    x[1, 0, 8999] = -5.0                              # one token
    x[2, 0, torch.rand(V, generator=g) < 0.999] = -INF
    x[3] = torch.finfo(F32).min                       # a mask of the lowest value over everything
    x[4, 0, 100:] = torch.finfo(F32).min
    x[5, 0, 77], x[5, 0, 5000] = INF, INF
    x[6, 0, 8000] = float("nan")
    x[7, 0, 1], x[7, 0, 3] = float("nan"), INF
    x[8, 0, :] = torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)
    x[9, 0, :] = 1e-42 * torch.randn(V, generator=g)  # subnormal logits
    x[10] *= 1e30                                     # far apart
    x[11, 0, :4] = torch.tensor([3.0e38, 3.4e38, 3.4e38, -3.4e38])
    x[12, 0, ::2] = -INF
    for kind in ("none", "top_k", "top_p", "min_p", "all", "greedy"):
        u = torch.rand(B, 1, generator=g)
        lim = _limits(B, kind, g)
        tokens, probs = _call(x, u, *lim)
        _check(x, u, *lim, tokens, probs, f"special {kind}")
        assert tokens[0].item() == -1 and probs[0].item() == 0 and tokens[1].item() == 8999


def test_ends_of_the_limits(native):
    """Limits beyond their ranges, infinite and NaN ones, uniform numbers at
    their ends."""
    g = torch.Generator().manual_seed(9)
    V, nan = 3001, float("nan")
    T = [1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, -1.0, nan, INF, INF, 1e-5, 9e-6, 3e38, 1.0, 1.0]
    k = [-3, 2 ** 62, V, V - 1, 0, 0, 0, 0, 0, 0, 0, 3000, 0, 0, 0, 0, 0]
    p = [1.0, 1.0, 1.0, 1.0, 2.0, nan, -1.0, 0.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1 - 2.0 ** -24]
    m = [0.0, 0.0, 0.0, 0.0, -1.0, nan, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 7.0, 0.0]
    B = len(T)
    x = torch.randn(B, 4, V, generator=g)
    u = torch.rand(B, 4, generator=g)
    u[:, 1], u[:, 2], u[:, 3] = 0.0, 1.0 - 2.0 ** -24, 5.0
    u[3, 3], u[4, 3] = -1.0, nan
    f = lambda a: [np.float32(v).item() for v in a]
    tokens, probs = _call(x, u, T, k, p, m)
    ur = torch.nan_to_num(u, nan=0.0)
    _check(x, ur, f(T), k, f(p), f(m), tokens, probs, "ends")


def test_numbers_for_all_requests_views_workspace(native):
    g = torch.Generator().manual_seed(10)
    B, M, V = 5, 3, 10001
    x = (2 * torch.randn(B, M, V, generator=g)).cuda()
    u = torch.rand(B, M, generator=g).cuda()
    want = _call(x, u, [np.float32(0.7).item()] * B, [30] * B, [np.float32(0.9).item()] * B, [np.float32(0.01).item()] * B)
    ws = rmd.Workspace(B, M, V, 1, sample=False, filtered=True)
    ws.buffer[131072:].fill_(0xFF)                        # the scratch needs no zero fill
    for kw in (dict(), dict(workspace=ws)):
        got = rmd.sample_block_filtered(x, u, 0.7, top_k=30, top_p=0.9, min_p=0.01, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    wide = torch.zeros(B, M, V + 9, device="cuda")
    wide[..., 4:V + 4] = x
    got = rmd.sample_block_filtered(wide[..., 4:V + 4], u.double(), torch.full((B,), 0.7, dtype=torch.float64).cuda(),
                                    top_k=torch.full((B,), 30, dtype=torch.int32).cuda(), top_p=0.9, min_p=0.01)
    assert torch.equal(got[0], want[0])
    # a batch split across calls is the whole one
    parts = [rmd.sample_block_filtered(x[b:b + 1, j:j + 1], u[b:b + 1, j:j + 1], 0.7, top_k=30, top_p=0.9, min_p=0.01)
             for b in range(B) for j in range(M)]
    assert torch.equal(torch.cat([t for t, _ in parts]).view(B, M), want[0])
    assert rmd.sample_block_filtered(x[:0], u[:0], 0.7)[0].shape == (0, M)
    # no temperature, as elsewhere: the largest logit
    got = rmd.sample_block_filtered(x, u, None, top_k=torch.tensor([3] * B).cuda())
    assert torch.equal(got[0], x.argmax(-1)) and bool((got[1] == 1).all())


def test_streams_and_graph(native):
    g = torch.Generator().manual_seed(12)
    B, M, V = 7, 2, 20000
    x = (2 * torch.randn(B, M, V, generator=g)).cuda()
    u = torch.rand(B, M, generator=g).cuda()
    lim = _limits(B, "mixed", g)
    dev = [torch.tensor(lim[0], dtype=F32).cuda(), torch.tensor(lim[1]).cuda(), torch.tensor(lim[2], dtype=F32).cuda(),
           torch.tensor(lim[3], dtype=F32).cuda()]
    ws = rmd.Workspace(B, M, V, 1, sample=False, filtered=True)

    def call(**kw):
        return rmd.sample_block_filtered(xs, us, dev[0], top_k=dev[1], top_p=dev[2], min_p=dev[3], **kw)

    xs, us = x.clone(), u.clone()
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = call(workspace=ws)
    for seed in range(3):
        xs.copy_(torch.randn(B, M, V, generator=g))
        us.copy_(torch.rand(B, M, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        want = call(workspace=ws)                          # eager, on the same workspace
        assert torch.equal(res[0], want[0]) and torch.equal(res[1], want[1])


def test_serving_step(native):
    """Logits by the 4-bit head, the request's rules, then its limits: every
    token from the rows it was drawn from, and none that the grammar forbids."""
    g = torch.Generator().manual_seed(13)
    B, M, V, d = 4, 3, 5000, 256
    hidden = torch.randn(B, M, d, generator=g).cuda()
    hc, hs = rmd.quantize_blocks_fp4((0.2 * torch.randn(V, d, generator=g)).cuda())
    allowed = torch.rand(B, M, V, generator=g) < 0.3
    allowed[3, 2] = False
    from tests import rules_reference as rules
    mask = torch.from_numpy(rules.pack_mask(allowed.numpy())).cuda()
    history = torch.randint(0, V, (B, 50), generator=g).cuda()
    base = rmd.lm_head_logits_fp4(hidden, hc, hs)
    logits = rmd.process_block_logits(base, history=history, repetition_penalty=torch.full((B,), 1.2).cuda(), token_mask=mask)
    u = torch.rand(B, M, generator=g)
    lim = _limits(B, "all", g)
    tokens, probs = _call(logits, u, *lim)
    _check(logits.cpu(), u, *lim, tokens, probs, "serving")
    t = tokens.cpu()
    assert t[3, 2] == -1
    at = t >= 0
    assert allowed[at].gather(1, t[at][:, None]).all()


def test_draws_follow_the_distribution(native):
    """A thousand evenly spread uniform numbers give every token as often as
    its probability says, to one."""
    V, n = 40, 1000
    g = torch.Generator().manual_seed(14)
    row = torch.randn(V, generator=g)
    u = (torch.arange(n, dtype=F32) + 0.5) / n
    tokens, _ = rmd.sample_block_filtered(row.expand(1, n, V).cuda(), u.view(1, n).cuda(), 0.8)
    got = torch.bincount(tokens.view(-1).cpu(), minlength=V).double()
    want = torch.softmax(row.double() / 0.8, 0) * n
    assert (got - want).abs().max() <= 1.0
