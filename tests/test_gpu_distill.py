"""Distillation from a teacher's top logits on the GPU against 64 bits."""
import numpy as np
import pytest
import torch

import rank_markov_draft_amd as rmd
from tests import distill_reference as ref
from tests import rules_reference as rules

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _inputs(B, M, V, K, dtype, tdtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = (2 * torch.randn(B, M, V, generator=g)).to(dtype)
    ids = torch.randint(0, V, (B, M, K), generator=g)
    t = (3 * torch.randn(B, M, K, generator=g)).to(tdtype)
    gl = torch.rand(B, M, generator=g) + 0.1
    return x, ids, t, gl


def _run(x, ids, t, gl, tau, **kw):
    xc, ic, tc = x.cuda(), ids.cuda(), t.cuda()
    loss, stats = rmd.distill_block_loss(xc, ic, tc, temperature=tau, **kw)
    grad = rmd.distill_block_loss_backward(gl.cuda(), xc, ic, tc, stats, temperature=tau)
    return loss, grad, stats


def _check(x, ids, t, gl, tau, loss, grad, what):
    wl, tl, wg, tg = ref.block(x.double().numpy(), ids.numpy(), t.double().numpy(), tau, gl.double().numpy())
    rules.check(loss, wl, tl, what + " loss")
    rules.check(grad, wg, tg, what + " gradient")


@pytest.mark.parametrize("dtype,tdtype", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("B,M,V,K,tau", [(1, 1, 1, 1, 1.0), (1, 1, 2, 5, 0.5), (2, 3, 7, 3, 2.0), (1, 2, 257, 300, 1.0),
                                         (3, 2, 2048, 20, 1.0), (2, 2, 8191, 17, 3.0), (1, 3, 8193, 64, 0.7),
                                         (1, 1, 50257, 1024, 1.0), (2, 1, 32000, 1, 1.0), (40, 3, 1001, 8, 1.0)])
def test_loss_and_gradient(native, B, M, V, K, tau, dtype, tdtype):
    """Random ids: lists with the same id more than once among them."""
    x, ids, t, gl = _inputs(B, M, V, K, dtype, tdtype, B + 7 * M + V + K)
    loss, grad, stats = _run(x, ids, t, gl, tau)
    assert loss.dtype == F32 and tuple(loss.shape) == (B, M) and tuple(stats.shape) == (B, M, 4) and grad.dtype == dtype
    _check(x, ids, t, gl, tau, loss, grad, f"{B}x{M} V {V} K {K}")


@pytest.mark.parametrize("rows", [1, 2, 300, 2100])
def test_slices(native, rows):
    """Rows cut into many slices, into a few, and one to a workgroup."""
    V = 40000 if rows < 100 else 17001 if rows < 1000 else 9001
    x, ids, t, gl = _inputs(rows, 1, V, 6, BF16, F32, rows)
    loss, grad, _ = _run(x, ids, t, gl, 1.0)
    at = sorted({0, 1 % rows, rows // 2, rows - 1})
    _check(x[at], ids[at], t[at], gl[at], 1.0, loss[at], grad[at], f"rows {rows}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lists_with_padding_and_masks(native, dtype):
    B, M, V, K = 3, 4, 5000, 9
    x, ids, t, gl = _inputs(B, M, V, K, dtype, F32, 5)
    ninf = float("-inf")
    ids[0, 0] = -1                                   # no entries
    ids[0, 1, 3:] = -1                               # a short list
    ids[0, 2, :3] = torch.tensor([V, 2 ** 40, -2 ** 62])
    t[0, 3, 2:5] = ninf                              # entries without weight
    t[1, 0] = ninf                                   # nothing but those
    ids[1, 1] = 77                                   # one id nine times
    x[1, 2] = ninf                                   # a row that a mask leaves nothing of
    x[1, 3] = ninf
    x[1, 3, 4321] = 2.0                              # and one with a single token left
    ids[1, 3, 0] = 4321
    x[2, 0, ::2] = ninf                              # masked tokens, some in the list
    ids[2, 0] = torch.arange(1, 2 * K, 2)
    x[2, 1] = torch.finfo(dtype).min                 # a mask of the type's lowest value over everything
    x[2, 2, 10:] = torch.finfo(dtype).min
    ids[2, 2] = torch.arange(K)
    t[2, 3] = torch.tensor([0.0, -1e30, -3e38, 5.0, -200.0, -100.0, 1.0, 2.0, 3.0])
    loss, grad, _ = _run(x, ids, t, gl, 1.0)
    _check(x, ids, t, gl, 1.0, loss, grad, "masks")
    assert loss[0, 0] == 0 and not grad[0, 0].any() and loss[1, 0] == 0 and not grad[1, 0].any()
    assert torch.isinf(loss[1, 2]) and not grad[1, 2].any()
    assert torch.isinf(loss[1, 3]) and torch.isfinite(grad[1, 3]).all()


def test_not_numbers_show_in_their_row(native):
    B, M, V, K = 1, 6, 3000, 4
    x, ids, t, gl = _inputs(B, M, V, K, F32, F32, 8)
    x[0, 1, 100] = float("nan")
    x[0, 2, 2999] = float("inf")
    t[0, 3, 1] = float("nan")
    t[0, 4, 1] = float("inf")
    ids[0, 5], t[0, 5, 2] = -1, float("nan")         # not an entry
    loss, grad, _ = _run(x, ids, t, gl, 1.0)
    assert torch.isnan(loss[0, 1:5]).all() and torch.isfinite(loss[0, 0]) and loss[0, 5] == 0
    assert torch.isnan(grad[0, 1]).all() and torch.isnan(grad[0, 2]).all() and not grad[0, 5].any()
    for m in (3, 4):
        nan = torch.isnan(grad[0, m])
        want = torch.zeros(V, dtype=torch.bool)
        want[ids[0, m]] = True
        assert torch.equal(nan.cpu(), want)


def test_gradient_against_differences(native):
    """The gradient against differences of the 64-bit loss."""
    tau, h = 1.5, 1e-4
    x, ids, t, gl = _inputs(1, 2, 600, 12, F32, F32, 11)
    _, grad, _ = _run(x, ids, t, gl, tau)
    X, T = x.double().numpy(), t.double().numpy()
    _, _, _, tol = ref.block(X, ids.numpy(), T, tau, gl.double().numpy())
    for m in range(2):
        for v in list(ids[0, m].numpy()) + list(range(0, 600, 37)):
            up, down = X[0, m].copy(), X[0, m].copy()
            up[v] += h
            down[v] -= h
            g = gl[0, m].item()
            diff = g * (ref.row(up, ids[0, m].numpy(), T[0, m], tau, g)[0] - ref.row(down, ids[0, m].numpy(), T[0, m], tau, g)[0]) / (2 * h)
            # a central difference is off by h^2 / 6 times the third derivative
            # (p's third cumulant, below 1/8, over tau), and 64-bit rounding over h
            assert abs(grad[0, m, v].item() - diff) <= tol[0, m, v] + g * h * h + 1e-10


def test_in_place_views_workspace_and_empty(native):
    x, ids, t, gl = (a.cuda() for a in _inputs(4, 3, 9001, 10, BF16, F32, 3))
    ids[0, 0, :4] = 9000                             # the row's last column
    loss, stats = rmd.distill_block_loss(x, ids, t)
    grad = rmd.distill_block_loss_backward(gl, x, ids, t, stats)
    ws = rmd.Workspace(4, 3, 9001, 1, sample=False, distill=True)
    ws.buffer[131072:].fill_(0xFF)                   # the scratch needs no zero fill
    l2, s2 = rmd.distill_block_loss(x, ids.to(torch.int32), t, workspace=ws)
    assert torch.equal(l2, loss) and torch.equal(s2, stats)
    wide = torch.zeros(4, 3, 9010, dtype=BF16, device="cuda")
    wide[..., :9001] = x
    l2, s2 = rmd.distill_block_loss(wide[..., :9001], ids, t)
    assert torch.equal(l2, loss) and torch.equal(s2, stats)
    y = x.clone()
    assert rmd.distill_block_loss_backward(gl, y, ids, t, stats, out=y) is y and torch.equal(y, grad)
    assert rmd.distill_block_loss(x[:0], ids[:0], t[:0])[0].shape == (0, 3)
    l0, s0 = rmd.distill_block_loss(x, ids[..., :0], t[..., :0])
    assert not l0.any() and not rmd.distill_block_loss_backward(gl, x, ids[..., :0], t[..., :0], s0).any()


def test_streams_and_graph(native):
    x, ids, t, gl = (a.cuda() for a in _inputs(5, 2, 20000, 16, F32, F32, 4))
    ws = rmd.Workspace(5, 2, 20000, 1, sample=False, distill=True)

    def step(x):
        loss, stats = rmd.distill_block_loss(x, ids, t, workspace=ws)
        return loss, rmd.distill_block_loss_backward(gl, x, ids, t, stats)

    want = step(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(x)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    xs = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(xs)
    for seed in range(3):
        xs.copy_(_inputs(5, 2, 20000, 16, F32, F32, 30 + seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = [r.clone() for r in res]
        want = step(xs)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_training_step_through_the_head(native):
    """Base logits by the 4-bit head, the Markov bias, the loss, its gradient
    and the gradients of W1 and W2: against the formulas in 64 bits and
    against differences of the loss."""
    B, M, V, d, r, K, tau = 2, 3, 700, 192, 16, 12, 1.3
    g = torch.Generator().manual_seed(21)
    hidden = torch.randn(B, M, d, generator=g).cuda()
    hc, hs = rmd.quantize_blocks_fp4((0.1 * torch.randn(V, d, generator=g)).cuda())
    w1, w2 = ((0.3 * torch.randn(V, r, generator=g)) for _ in range(2))
    prev = torch.randint(0, V, (B, M), generator=g)
    _, ids, t, gl = _inputs(B, M, V, K, F32, F32, 22)
    base = rmd.lm_head_logits_fp4(hidden, hc, hs)
    corrected = rmd.apply_block_logits(base, prev.cuda(), w1.cuda(), w2.cuda())
    loss, stats = rmd.distill_block_loss(corrected, ids.cuda(), t.cuda(), temperature=tau)
    grad = rmd.distill_block_loss_backward(gl.cuda(), corrected, ids.cuda(), t.cuda(), stats, temperature=tau)
    gw1, gw2 = rmd.apply_block_logits_backward(grad, prev.cuda(), w1.cuda(), w2.cuda())
    # from the kernel's own corrected logits on
    wl, tl, wg, tg = ref.block(corrected.cpu().double().numpy(), ids.numpy(), t.double().numpy(), tau, gl.double().numpy())
    rules.check(loss, wl, tl, "loss")
    W1, W2, P = w1.double().numpy(), w2.double().numpy(), prev.numpy().reshape(-1)
    G, TG = wg.reshape(-1, V), tg.reshape(-1, V) + 2.0 ** -24 * np.abs(wg.reshape(-1, V))
    d1, t1 = np.zeros((V, r)), np.zeros((V, r))
    for n in range(B * M):
        d1[P[n]] += G[n] @ W2
        # fp32 sums of V products, worst order, over all rows of an id
        t1[P[n]] += (TG[n] + (V + B * M) * 2.0 ** -24 * np.abs(G[n])) @ np.abs(W2)
    d2 = G.T @ W1[P]
    t2 = (TG + (B * M + 2) * 2.0 ** -24 * np.abs(G)).T @ np.abs(W1[P])
    rules.check(gw1, d1, t1, "gradient of W1")
    rules.check(gw2, d2, t2, "gradient of W2")
    # and differences of the whole loss in 64 bits, from the base logits
    b64 = base.cpu().double().numpy().reshape(-1, V)

    def total(W1, W2):
        x = b64 + W1[P] @ W2.T
        return sum(gl.reshape(-1)[n].item() * ref.row(x[n], ids.numpy().reshape(-1, K)[n], t.double().numpy().reshape(-1, K)[n],
                                                      tau, 1.0)[0] for n in range(B * M))

    h = 1e-4
    rng = np.random.default_rng(1)
    for i, j in zip(rng.integers(0, V, 20), rng.integers(0, r, 20)):
        for W, got in ((0, gw1), (1, gw2)):
            at = (P[i % P.size], j) if W == 0 else (i, j)
            ws = []
            for s in (h, -h):
                pair = [W1.copy(), W2.copy()]
                pair[W][at] += s
                ws.append(total(*pair))
            # the corrected logits' own rounding (2^-24 of up to 16, three roundings) moves p and q by that much
            tol = 1e-6 * (1 + np.abs(G).sum()) + h * h * 10
            assert abs(got[at].item() - (ws[0] - ws[1]) / (2 * h)) <= tol
