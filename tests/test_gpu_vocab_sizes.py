"""The 4-bit head at every tile size, and the 4-bit head, sampling under limits
and the distillation loss past one launch's workgroups, past 2^32 elements and
at the largest vocabularies."""
import numpy as np
import pytest
import torch

import rank_markov_draft_amd as rmd
from tests import blocks_reference as ref
from tests import rules_reference as rules

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def room(native):
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    return dict(device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


# ------------------------------------------------------------ 4-bit head
# on 256 CUs: tiles of 32 x 128, 64 x 128, 64 x 256, 128 x 256, twice 320 x 192, 256
# x 256, 320 x 128, again 320 x 192, and 192 x 256; d ends in half a chunk, a third of its last
# group of blocks filled
@pytest.mark.parametrize("odt", [F32, BF16])
@pytest.mark.parametrize("rows,V", [(1, 70001), (40, 70001), (40, 129280), (70, 70001), (130, 70001), (200, 70001), (700, 70001),
                                    (650, 6983), (300, 129280), (330, 129280)])
def test_head_tiles(native, rows, V, odt):
    d = 556
    x = torch.randn(rows, d, **_gen(rows))
    w = 0.05 * torch.randn(V, d, **_gen(V))
    hc, hs = rmd.quantize_blocks_fp4(w)
    got = rmd.lm_head_logits_fp4(x, hc, hs, out_dtype=odt)
    a = ref.values(*ref.quantize(x.cpu().numpy()))
    cols = np.unique(np.r_[np.arange(0, V, 61), np.arange(V - 330, V)])
    at = torch.from_numpy(cols).cuda()
    b = ref.values(ref.unpack(hc[at].cpu().numpy()), hs[at].cpu().numpy())
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    # two roundings of at most a step (2^-23) a matrix instruction of 64 numbers
    rules.check(got[:, at], want, 2 * ((d + 63) // 64) * 2.0 ** -23 * size, f"rows {rows} V {V}")
    # whole rows against the same product of values
    wq = rmd.dequantize_blocks_fp4(hc, hs, d)
    full = torch.from_numpy(a[:, :d]).float().cuda() @ wq.t()
    assert (got.float() - full).abs().max() <= 0.01 * full.abs().max() + 1e-4


def test_head_past_32_bits(native):
    """Codes past 2^32 bytes, logits past 2^32 elements."""
    V, d, rows = 2 ** 26 + 77, 128, 65
    hc = torch.randint(0, 256, (V, 64), dtype=torch.uint8, **_gen(1))
    hs = torch.randint(118, 124, (V, 4), dtype=torch.uint8, **_gen(2))
    x = torch.randn(rows, d, **_gen(3)).to(BF16)
    got = rmd.lm_head_logits_fp4(x, hc, hs, out_dtype=BF16)
    for a, b in ((0, 1000), (2 ** 25, 2 ** 25 + 1000), (V - 1003, V)):
        want = rmd.lm_head_logits_fp4(x, hc[a:b].clone(), hs[a:b].clone(), out_dtype=BF16)
        assert torch.equal(got[:, a:b], want)
    n = 1 << 22
    for a in range(0, V, n):                         # every column was written
        assert bool((got[:, a:a + n] != 0).any(0).all())


def test_quantize_past_32_bits(native):
    rows, d = 2 ** 24 + 3, 288
    x = torch.randn(rows, d, dtype=BF16, **_gen(4))
    codes, scales = rmd.quantize_blocks_fp4(x)
    y = rmd.dequantize_blocks_fp4(codes, scales, d, dtype=BF16)
    for a, b in ((0, 9), (rows // 2, rows // 2 + 9), (rows - 9, rows)):
        wc, ws = rmd.quantize_blocks_fp4(x[a:b].clone())
        assert torch.equal(codes[a:b], wc) and torch.equal(scales[a:b], ws)
        assert torch.equal(y[a:b], rmd.dequantize_blocks_fp4(wc, ws, d, dtype=BF16))
    n = 1 << 20
    for a in range(0, rows, n):                      # within half a step of the block's largest everywhere
        part = x[a:a + n].float()
        assert bool(((y[a:a + n].float() - part).abs() <= part.abs().amax(-1, keepdim=True) / 4).all())


# ------------------------------------------------------------ sampling
def test_sample_more_rows_than_a_launch(native):
    """A workgroup of 512 a row: 2^23 - 1 rows a launch."""
    rows, V = 2 ** 23 + 9, 9
    x = torch.randn(rows, 1, V, dtype=BF16, **_gen(5))
    u = torch.rand(rows, 1, **_gen(6))
    k = torch.randint(0, 10, (rows,), **_gen(7))
    p = torch.rand(rows, **_gen(8))
    t, q = rmd.sample_block_filtered(x, u, 0.8, top_k=k, top_p=p)
    for a, b in ((0, 9), (2 ** 23 - 9, 2 ** 23 + 2), (rows - 9, rows)):
        wt, wq = rmd.sample_block_filtered(x[a:b].clone(), u[a:b].clone(), 0.8, top_k=k[a:b].clone(), top_p=p[a:b].clone())
        assert torch.equal(t[a:b], wt) and torch.equal(q[a:b], wq)
    assert bool(((t >= 0) & (t < V)).all()) and bool(((q > 0) & (q <= 1)).all())


def test_sample_past_32_bits(native):
    V, B = 2 ** 27 + 5, 33
    x = torch.randn(B, 1, V, dtype=BF16, **_gen(9))
    u = torch.rand(B, 1, **_gen(10))
    kind = torch.arange(B, device="cuda") % 3
    kw = dict(top_k=torch.where(kind == 0, 40, 0), top_p=torch.where(kind == 1, 0.7, 1.0))
    t, q = rmd.sample_block_filtered(x, u, 1.0, **kw)
    for b in (0, 1, 2, 30, 31, 32):
        wt, wq = rmd.sample_block_filtered(x[b:b + 1].clone(), u[b:b + 1], 1.0, **{n: v[b:b + 1] for n, v in kw.items()})
        assert torch.equal(t[b], wt[0]) and torch.equal(q[b], wq[0])


@pytest.mark.parametrize("V", [2 ** 30, 2 ** 30 - 5])
def test_sample_largest_vocabulary(native, V):
    """Four tokens above the rest, at both ends and in between."""
    x = torch.full((1, 1, V), -40.0, dtype=BF16, device="cuda")
    at = [5, V // 2 + 1, V - 4, V - 1]
    for v in at:
        x[0, 0, v] = 3.0
    u = torch.tensor([[0.0]], device="cuda")
    for i, v in enumerate(at):
        u[0, 0] = (i + 0.5) / 4
        for kw in (dict(top_k=4), dict(top_p=0.99999), dict(min_p=0.5), dict()):
            t, q = rmd.sample_block_filtered(x, u, 0.5, **kw)
            assert t.item() == v and q.item() == 0.25, (i, kw)
    assert rmd.sample_block_filtered(x, u, 0.0)[0].item() == 5
    # all tokens alike, kept up to a border far behind
    x.fill_(1.0)
    u[0, 0] = 0.5
    t, q = rmd.sample_block_filtered(x, u, 1.0, top_k=V // 2)
    assert t.item() == V // 4 and q.item() == np.float32(1 / (V // 2)).item()
    t, q = rmd.sample_block_filtered(x, u, 1.0, top_p=0.5)
    n = -(-V // 2)
    assert t.item() == n // 2 and q.item() == np.float32(1 / n).item()


# ------------------------------------------------------------ distillation
def test_distill_more_rows_than_a_launch(native):
    """A workgroup of 256 a row: 2^24 - 1 rows a launch."""
    rows, V, K = 2 ** 24 + 9, 5, 2
    x = torch.randn(rows, 1, V, dtype=BF16, **_gen(11))
    ids = torch.randint(-1, V, (rows, 1, K), **_gen(12))
    t = torch.randn(rows, 1, K, **_gen(13))
    g = torch.rand(rows, 1, **_gen(14)) + 0.5
    loss, st = rmd.distill_block_loss(x, ids, t)
    grad = rmd.distill_block_loss_backward(g, x, ids, t, st)
    for a, b in ((0, 9), (2 ** 24 - 9, 2 ** 24 + 2), (rows - 9, rows)):
        wl, ws = rmd.distill_block_loss(x[a:b].clone(), ids[a:b].clone(), t[a:b].clone())
        assert torch.equal(loss[a:b], wl) and torch.equal(st[a:b], ws)
        assert torch.equal(grad[a:b], rmd.distill_block_loss_backward(g[a:b].clone(), x[a:b].clone(), ids[a:b].clone(),
                                                                      t[a:b].clone(), ws))
    some = (ids >= 0).any(-1)
    assert bool((loss[~some] == 0).all()) and bool(torch.isfinite(loss).all()) and bool(torch.isfinite(grad).all())
    # where no id stands twice sum q (log q - log p) >= 0; twice the same id with
    # q = (1/2, 1/2) gives log(1/2) - log p, which is below 0 for p > 1/2
    once = some & (ids[..., 0] != ids[..., 1])
    assert bool((loss[once] > -1e-6).all())


@pytest.mark.parametrize("B,V", [(33, 2 ** 27 + 5), (1, 2 ** 30)])
def test_distill_past_32_bits(native, B, V):
    x = torch.randn(B, 1, V, dtype=BF16, **_gen(15))
    ids = torch.randint(0, V, (B, 1, 4), **_gen(16))
    ids[:, :, 0] = V - 1
    t = torch.randn(B, 1, 4, **_gen(17))
    g = torch.rand(B, 1, **_gen(18)) + 0.5
    loss, st = rmd.distill_block_loss(x, ids, t)
    grad = rmd.distill_block_loss_backward(g, x, ids, t, st)
    for b in sorted({0, B // 2, B - 1}):
        xb = x[b, 0].double()
        top = xb.max()
        z = torch.exp(xb - top).sum()
        q = torch.softmax(t[b, 0].double(), 0)
        logp = xb[ids[b, 0]] - top - torch.log(z)
        want = (q * (torch.log(q) - logp)).sum()
        # the streamed sum's worst case is far off its usual one; V / 2^27 terms a lane and slice
        assert abs(loss[b, 0].double() - want) <= 1e-5 * (1 + want)
        cols = torch.randint(0, V, (1000,), **_gen(19))
        p = torch.exp(xb[cols] - top) / z * g[b, 0].double()
        hit = torch.isin(cols, ids[b, 0])
        assert bool(((grad[b, 0, cols].double() - p).abs()[~hit] <= (2.0 ** -8 + 1e-4) * p[~hit] + 2.0 ** -126).all())
        for j in range(4):
            w = (torch.exp(logp[j]) - q[ids[b, 0] == ids[b, 0, j]].sum()) * g[b, 0].double()
            assert abs(grad[b, 0, ids[b, 0, j]].double() - w) <= 2.0 ** -8 * abs(w) + 1e-6
        del xb
