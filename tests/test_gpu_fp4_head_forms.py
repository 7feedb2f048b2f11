"""Every form of the 4-bit head's kernel (tiles of 32 x 128 to 320 x 192 on 256
compute units) where its chunk stream is at its ends: rows that end inside a chunk
next to rows with NaN scales, one chunk a tile with several tiles a workgroup, and
the long stream of d = 5120."""
import numpy as np
import pytest
import torch

import rank_markov_draft_amd as rmd
from tests import blocks_reference as ref


F32, BF16 = torch.float32, torch.bfloat16
# rows and vocabulary of more tiles than compute units, by tile
FORMS = {"32x128": (1, 70001), "64x128": (40, 70001), "64x256": (40, 129280), "128x256": (70, 70001), "192x256": (330, 129280),
         "256x256": (700, 70001), "320x128": (300, 50021), "320x192": (130, 70001), "320x192 twice": (330, 70001)}
pytestmark = [pytest.mark.gpu, pytest.mark.parametrize("rows,V", list(FORMS.values()), ids=list(FORMS))]


@pytest.fixture(autouse=True)
def room(native):
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    return dict(device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


def _check_whole(got, x, hc, hs, d, what):
    """All logits against an fp32 product of the numbers that both sides stand
    for; columns that stand for NaN are the caller's."""
    a = torch.from_numpy(ref.values(*ref.quantize(x.float().cpu().numpy()))[:, :d]).float().cuda()
    w = rmd.dequantize_blocks_fp4(hc, hs, d)
    want, size = a @ w.t(), a.abs() @ w.abs().t()
    # the head: two roundings of at most a step (2^-23) of what has been added up
    # for a matrix instruction of 64 numbers; the product: half a step (2^-24) for
    # each of d products and sums; the size itself may be as much too small
    tol = (2 * ((d + 63) // 64) * 2.0 ** -23 + 2 * d * 2.0 ** -24) * (1 + d * 2.0 ** -23) * size
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert bool(((got.float() - want).abs() <= tol).all()), what


def _check_columns(got, x, hc, hs, cols, what):
    """Some columns against 64 bits."""
    a = ref.values(*ref.quantize(x.float().cpu().numpy()))
    at = torch.from_numpy(cols).cuda()
    b = ref.values(ref.unpack(hc[at].cpu().numpy()), hs[at].cpu().numpy())
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = 2 * ((x.shape[-1] + 63) // 64) * 2.0 ** -23 * size
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    assert (np.abs(got[:, at].double().cpu().numpy() - want) <= tol).all(), what


def _columns(V):
    return np.unique(np.r_[np.arange(0, V, 211), np.arange(V - 400, V)])


@pytest.mark.parametrize("odt", [F32, BF16])
@pytest.mark.parametrize("d", [300, 4900])
def test_not_numbers_stay_in_their_row_and_channel(native, rows, V, d, odt):
    """Both d end in half a chunk, whose other half in LDS holds the first
    blocks of the next row: there NaN scales stand, at tiles' ends too."""
    x = torch.randn(rows, d, **_gen(rows))
    w = 0.02 * torch.randn(V, d, **_gen(V))
    bad_rows = [] if rows == 1 else [r for r in (1, 31, 32, 63, 64, 127, 128, 192, 255, 256, 319, 320, rows - 1) if r < rows]
    for i, r in enumerate(bad_rows):
        x[r, (0, 40, d - 1)[i % 3]] = (float("nan"), float("inf"))[i % 2]
    bad = np.unique(np.r_[np.arange(7, V, 1001), 127, 128, 191, 192, 255, 256, 383, 384, 512, V - 1])
    for i, v in enumerate(bad):
        w[int(v), (0, 3, 33, d - 1)[i % 4]] = (float("inf"), float("nan"), -float("inf"))[i % 3]
    hc, hs = rmd.quantize_blocks_fp4(w)
    got = rmd.lm_head_logits_fp4(x, hc, hs, out_dtype=odt)
    want = torch.zeros(rows, V, dtype=torch.bool, device="cuda")
    want[:, torch.from_numpy(bad).cuda()] = True
    want[bad_rows] = True
    assert torch.equal(torch.isnan(got), want)
    good_rows = torch.tensor([r for r in range(rows) if r not in bad_rows], device="cuda")
    cols = np.setdiff1d(_columns(V), bad)
    _check_columns(got[good_rows], x[good_rows], hc, hs, cols, f"rows {rows} V {V} d {d}")


@pytest.mark.parametrize("odt", [F32, BF16])
@pytest.mark.parametrize("d", [33, 128, 200, 256])
def test_one_chunk_a_tile(native, rows, V, d, odt):
    """The wait for a tile's only chunk counts the stores of the one before."""
    x = torch.randn(rows, d, **_gen(rows + d)).to(BF16)
    hc, hs = rmd.quantize_blocks_fp4(0.1 * torch.randn(V, d, **_gen(V + d)))
    got = rmd.lm_head_logits_fp4(x, hc, hs, out_dtype=odt)
    _check_whole(got, x, hc, hs, d, f"rows {rows} V {V} d {d}")
    _check_columns(got, x, hc, hs, _columns(V), f"rows {rows} V {V} d {d}")


@pytest.mark.parametrize("odt", [F32, BF16])
def test_long_rows(native, rows, V, odt):
    d = 5120
    x = torch.randn(rows, d, **_gen(rows)).to(BF16)
    hc = torch.empty(V, d // 2, dtype=torch.uint8, device="cuda")
    hs = torch.empty(V, d // 32, dtype=torch.uint8, device="cuda")
    for a in range(0, V, 1 << 15):
        n = min(V, a + (1 << 15)) - a
        rmd.quantize_blocks_fp4(0.02 * torch.randn(n, d, **_gen(a)), out=hc[a:a + n], scale_out=hs[a:a + n])
    got = rmd.lm_head_logits_fp4(x, hc, hs, out_dtype=odt)
    _check_whole(got, x, hc, hs, d, f"rows {rows} V {V}")
    _check_columns(got, x, hc, hs, _columns(V)[::3], f"rows {rows} V {V}")
