"""Microscaled 4-bit blocks and the vocabulary head held in them, on the GPU
against 64 bits: codes, scales and the numbers they stand for equal, logits
within the roundings of the matrix cores' sums and of the output type."""
import numpy as np
import pytest
import torch

import rank_markov_draft_amd as rmd
from tests import blocks_reference as ref
from tests import rules_reference as rules

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _rows(rows, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, d, generator=g) * torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g).float())
    return x.to(dtype)


def _check_blocks(x, codes, scales):
    wc, ws = ref.quantize(x.float().numpy().reshape(-1, x.shape[-1]))
    assert np.array_equal(scales.cpu().numpy().reshape(ws.shape), ws)
    got = ref.unpack(codes.cpu().numpy().reshape(wc.shape[0], -1))
    # both zeros stand for zero
    assert np.array_equal(np.where(got == 8, 0, got), np.where(wc == 8, 0, wc))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 31), (3, 32), (5, 33), (2, 127), (4, 128), (3, 129), (7, 264), (5, 500),
                                    (2, 2056), (70, 5120), (300, 64), (1, 8200), (3, 4099)])
def test_quantize(native, rows, d, dtype):
    x = _rows(rows, d, dtype, rows * 31 + d)
    codes, scales = rmd.quantize_blocks_fp4(x.cuda())
    n = ref.blocks_of(d)
    assert tuple(codes.shape) == (rows, 16 * n) and tuple(scales.shape) == (rows, n)
    _check_blocks(x, codes, scales)
    for out in (F32, BF16):
        y = rmd.dequantize_blocks_fp4(codes, scales, d, dtype=out).cpu()
        want = ref.values(*ref.quantize(x.float().numpy()))[:, :d]
        assert np.array_equal(y.double().numpy(), want)


def test_quantize_ties_and_ends(native):
    """Halves go to the even code, what lies above 6 to 6; the smallest and
    largest scales; zeros; infinities and NaN in one block alone."""
    x = torch.zeros(9, 96)
    x[0, :10] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -2.5])
    x[1, :5] = torch.tensor([7.9, 6.9, 5.1, 4.9, -7.0])
    x[2, :4] = torch.tensor([torch.finfo(F32).max, torch.finfo(F32).min, 1e38, 1.0])
    x[3, :3] = torch.tensor([2.0 ** -149, -2.0 ** -149, 0.0])
    x[4, :4] = torch.tensor([6 * 2.0 ** -127, -2.0 ** -127, 2.0 ** -128, 2.0 ** -129])
    x[5, :3] = torch.tensor([2.0 ** -126, 2.0 ** -125, 2.0 ** -124])
    x[6, 0], x[6, 40], x[6, 70] = 1.0, float("inf"), 2.0
    x[7, 5], x[7, 70] = float("nan"), -3.0
    x[8, 33:66] = torch.linspace(-8, 8, 33)
    codes, scales = rmd.quantize_blocks_fp4(x.cuda())
    _check_blocks(x, codes, scales)
    assert scales[6].tolist()[:3] == [125, 255, 126] and scales[7].tolist()[:3] == [255, 0, 126]
    y = rmd.dequantize_blocks_fp4(codes, scales, 96).cpu()
    want = ref.values(ref.unpack(codes.cpu().numpy()), scales.cpu().numpy())[:, :96]
    assert np.array_equal(y.double().numpy(), want, equal_nan=True)
    assert torch.isnan(y[6, 32:64]).all() and torch.isnan(y[7, :32]).all() and not torch.isnan(y[7, 32:]).any()


def test_views_outputs_and_empty(native):
    x = _rows(12, 160, F32, 5).cuda()
    codes, scales = rmd.quantize_blocks_fp4(x)
    c2, s2 = rmd.quantize_blocks_fp4(x.view(3, 4, 160))
    assert torch.equal(c2.view(12, -1), codes) and torch.equal(s2.view(12, -1), scales)
    ct, st = rmd.quantize_blocks_fp4(x.t())
    _check_blocks(x.t().cpu(), ct, st)
    odd = torch.empty(12 * 160 + 1, device="cuda")[1:].view(12, 160)     # rows that are no whole vectors
    odd.copy_(x)
    out, so = torch.empty_like(codes), torch.empty_like(scales)
    assert rmd.quantize_blocks_fp4(odd, out=out, scale_out=so) == (out, so)
    assert torch.equal(out, codes) and torch.equal(so, scales)
    y = rmd.dequantize_blocks_fp4(codes, scales, 160)
    back = torch.empty(12 * 160 + 1, device="cuda")
    back[0] = 7.0
    rmd.dequantize_blocks_fp4(codes, scales, 160, out=back[1:].view(12, 160))
    assert back[0] == 7.0 and torch.equal(back[1:].view(12, 160), y)
    assert rmd.quantize_blocks_fp4(x[:0])[0].shape == (0, 128) and rmd.quantize_blocks_fp4(x[:, :0])[1].shape == (12, 0)
    assert rmd.dequantize_blocks_fp4(codes[:0], scales[:0], 160).shape == (0, 160)
    shifted = torch.empty(codes.numel() + 1, dtype=torch.uint8, device="cuda")[1:].view_as(codes)
    shifted.copy_(codes)
    assert torch.equal(rmd.dequantize_blocks_fp4(shifted, scales, 160), y)


def _head(V, d, seed):
    codes, scales = ref.quantize(0.02 * np.random.default_rng(seed).standard_normal((V, d)).astype(np.float32))
    # what stands past d does not count: any codes of another row's would do
    return torch.from_numpy(ref.pack(codes)), torch.from_numpy(scales)


def _check_logits(got, x, hc, hs, what):
    d = x.shape[-1]
    a = ref.values(*ref.quantize(x.float().numpy()))
    b = ref.values(ref.unpack(hc.numpy()), hs.numpy())
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    # the products of two codes and their sum over a block are exact (below
    # 2^11, in quarters); a matrix instruction adds two blocks to the running
    # sum, two roundings of at most a step (2^-23) of what has been added up
    tol = 2 * ((d + 63) // 64) * 2.0 ** -23 * size
    rules.check(got.cpu().reshape(want.shape), want, tol, what)


@pytest.mark.parametrize("hdt,odt", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("rows,d,V", [(1, 1, 1), (1, 64, 33), (5, 100, 130), (31, 256, 257), (32, 288, 129), (33, 512, 300),
                                      (64, 640, 1000), (65, 129, 511), (130, 1000, 515), (200, 384, 777)])
def test_head(native, rows, d, V, hdt, odt):
    x = _rows(rows, d, hdt, rows + d + V)
    hc, hs = _head(V, d, V)
    got = rmd.lm_head_logits_fp4(x.cuda(), hc.cuda(), hs.cuda(), out_dtype=odt)
    assert got.dtype == odt and tuple(got.shape) == (rows, V)
    _check_logits(got, x, hc, hs, f"rows {rows} d {d} V {V}")


@pytest.mark.parametrize("rows", [1, 40, 129, 193, 257, 400, 700])
def test_head_tiles(native, rows):
    """Batches of every tile size, and a workgroup's second tile."""
    d, V = 416, 70001
    x = _rows(rows, d, BF16, rows)
    hc, hs = _head(V, d, rows)
    got = rmd.lm_head_logits_fp4(x.cuda(), hc.cuda(), hs.cuda(), out_dtype=F32)
    cols = np.unique(np.r_[np.arange(0, V, 97), np.arange(V - 300, V)])
    _check_logits(got[:, torch.from_numpy(cols).cuda()], x, hc[cols], hs[cols], f"rows {rows}")


@pytest.mark.parametrize("rows", [3, 70, 300])
def test_head_not_numbers_stay_in_their_row_and_channel(native, rows):
    """A NaN scale in a row of x or of the head shows in that row or channel
    alone, also next to a row that ends inside a chunk."""
    d, V = 300, 400
    x = _rows(rows, d, F32, 9)
    x[1, 40], x[2, 299] = float("nan"), float("inf")
    w = 0.02 * np.random.default_rng(1).standard_normal((V, d)).astype(np.float32)
    w[7, 3] = np.inf
    w[101, 280] = np.nan
    codes, scales = ref.quantize(w)
    hc, hs = torch.from_numpy(ref.pack(codes)), torch.from_numpy(scales)
    got = rmd.lm_head_logits_fp4(x.cuda(), hc.cuda(), hs.cuda()).cpu()
    nan = torch.isnan(got)
    want = torch.zeros(rows, V, dtype=torch.bool)
    want[1:3] = True
    want[:, [7, 101]] = True
    assert torch.equal(nan, want)
    _check_logits(got, x, hc, hs, "not numbers")


def test_head_views_outputs_workspace_streams_and_graph(native):
    d, V = 320, 1000
    x = _rows(24, d, BF16, 3).cuda()
    hc, hs = (t.cuda() for t in _head(V, d, 4))
    want = rmd.lm_head_logits_fp4(x, hc, hs)
    assert torch.equal(rmd.lm_head_logits_fp4(x.view(2, 3, 4, d), hc, hs).view(24, V), want)
    ws = rmd.Workspace(8, 5, V, 1, sample=False, fp4_hidden=d)
    ws.buffer[131072:].fill_(0xFF)                        # the scratch needs no zero fill
    out = torch.empty(25, V, device="cuda")
    out[24] = 5.0
    assert torch.equal(rmd.lm_head_logits_fp4(x, hc, hs, out=out[:24], workspace=ws), want) and bool((out[24] == 5.0).all())
    shifted = torch.empty(hc.numel() + 1, dtype=torch.uint8, device="cuda")[1:].view_as(hc)
    shifted.copy_(hc)
    assert torch.equal(rmd.lm_head_logits_fp4(x, shifted, hs), want)
    assert rmd.lm_head_logits_fp4(x[:0], hc, hs).shape == (0, V) and rmd.lm_head_logits_fp4(x, hc[:0], hs[:0]).shape == (24, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = rmd.lm_head_logits_fp4(x, hc, hs, out_dtype=F32)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(graph):
        res = rmd.lm_head_logits_fp4(xs, hc, hs, workspace=ws)
    for seed in range(3):
        xs.copy_(_rows(24, d, BF16, 50 + seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res, rmd.lm_head_logits_fp4(xs, hc, hs))


def test_head_equals_the_product_of_what_its_parts_stand_for(native):
    """quantize, dequantize and a plain product agree with the head where the
    sums are exact in fp32."""
    d, V = 256, 500
    g = torch.Generator().manual_seed(2)
    x, w = torch.randint(-6, 7, (20, d), generator=g).float(), torch.randint(-6, 7, (V, d), generator=g).float()
    hc, hs = rmd.quantize_blocks_fp4(w.cuda())
    xq = rmd.dequantize_blocks_fp4(*rmd.quantize_blocks_fp4(x.cuda()), d)
    wq = rmd.dequantize_blocks_fp4(hc, hs, d)
    assert torch.equal(rmd.lm_head_logits_fp4(x.cuda(), hc, hs), xq @ wq.t())
