"""The older entry points past one launch's 2^24 - 1 workgroups of 256: rows of
a sampled step, elements of the gate and of the backward."""
import pytest
import torch

import rank_markov_draft_amd as rmd

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
N = 2 ** 24 + 5


@pytest.fixture(autouse=True)
def room(native):
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    return dict(device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


def test_sampled_steps(native):
    V, r = 8, 4
    x = torch.randn(N, 2, V, **_gen(1))
    w1, w2 = (torch.randn(V, r, **_gen(2 + i)) for i in range(2))
    first = torch.randint(0, V, (N,), **_gen(4))
    tok, rows = rmd.sample_block_tokens(x, first, w1, w2, 0.7, seed=2)
    for a, b in ((0, 70), (2 ** 24 - 70, 2 ** 24 + 4), (N - 70, N)):
        t, o = rmd.sample_block_tokens(x[a:b], first[a:b], w1, w2, 0.7, seed=2, batch_offset=a)
        assert torch.equal(t, tok[a:b]) and torch.equal(o, rows[a:b])


def test_gate(native):
    """2^24 + 5 rows by 256 units, one thread each."""
    V, r, d = 8, 256, 1
    x = torch.randn(N, 1, V, dtype=BF16, **_gen(1))
    hidden = torch.randn(N, 1, d, dtype=BF16, **_gen(2))
    w1, w2, gw = (torch.randn(*s, **_gen(3 + i)).to(BF16) * 0.2 for i, s in enumerate(((V, r), (V, r), (r, d + r))))
    gb = torch.randn(r, **_gen(6)).to(BF16)
    ids = torch.randint(0, V, (N, 1), **_gen(7))
    out, latent = rmd.apply_block_logits_gated(x, ids, w1, w2, gw, gb, hidden, return_latent=True)
    for a, b in ((0, 70), (2 ** 24 - 70, 2 ** 24 + 4), (N - 70, N)):
        o, u = rmd.apply_block_logits_gated(x[a:b], ids[a:b], w1, w2, gw, gb, hidden[a:b], return_latent=True)
        assert torch.equal(u, latent[a:b]) and torch.equal(o, out[a:b])


def test_backward_of_a_long_vocabulary(native):
    """A weight gradient of 2^24 + 5 columns by 256 units, one thread each."""
    V, r = N, 256
    g = torch.randn(1, 2, V, **_gen(1)).to(BF16)
    w1 = torch.zeros(V, r, dtype=BF16, device="cuda")
    ids = torch.tensor([[3, V - 2]], device="cuda")
    w1[ids[0]] = torch.randn(2, r, **_gen(2)).to(BF16)
    gw1, gw2 = rmd.apply_block_logits_backward(g, ids, w1, torch.zeros_like(w1))
    assert not gw1.any()                             # W2 is zero
    e = w1[ids[0]].double()
    for a, b in ((0, 70), (2 ** 24 - 70, V)):
        want = g[0, :, a:b].double().t().contiguous() @ e
        # one rounding to bf16 of an fp32 sum of two products (compensated: each step within 2^-24 of its terms)
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -20 * (g[0, :, a:b].double().abs().t().contiguous() @ e.abs())
        assert ((gw2[a:b].double() - want).abs() <= tol).all()


def test_fp32_weights_past_2_30_columns(native):
    """Tiles of 128 columns by 512 threads end at 2^30 columns."""
    V, r = 2 ** 30 + 132, 4
    x = torch.zeros(1, 2, V, dtype=BF16, device="cuda")
    w1, w2 = (torch.zeros(V, r, device="cuda") for _ in range(2))
    ids = torch.tensor([[5, V - 1]], device="cuda")
    w1[ids[0]] = torch.tensor([[1.0, 2, 3, 4], [5, 6, 7, 8]], device="cuda")
    at = torch.tensor([0, 127, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 128, V - 1], device="cuda")
    w2[at] = torch.arange(24, device="cuda", dtype=F32).view(6, 4)
    x[:, :, 1], x[:, :, V - 2] = 3.0, 5.0
    out = rmd.apply_block_logits(x, ids, w1, w2)
    assert torch.equal(out[0][:, at], (w1[ids[0]].double().cpu() @ w2[at].double().cpu().t().contiguous()).to(BF16).cuda())
    assert out[0, 0, 1].item() == 3.0 and out[0, 1, V - 2].item() == 5.0
    out[:, :, at], out[:, :, 1], out[:, :, V - 2] = 0.0, 0.0, 0.0
    assert not out.any()
