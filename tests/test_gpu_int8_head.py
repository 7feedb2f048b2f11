"""The 8-bit vocabulary head on the GPU against 64 bits: integers equal, scales
equal, logits within the roundings of the scales' product, of the sum's
conversion, of their product and of the output type."""
import numpy as np
import pytest
import torch

import rank_markov_draft_amd as rmd
from tests import rules_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _rows(rows, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, d, generator=g).to(dtype)


def _head(V, d, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-127, 128, (V, d), generator=g).to(torch.int8)
    return q, torch.rand(V, generator=g) * 1e-3 + 1e-5


def _check_logits(got, x, hq, hs):
    q, s = ref.quantize(x.float().numpy())
    acc = q @ hq.numpy().astype(np.float64).T
    want = acc * s[:, None] * hs.numpy().astype(np.float64)[None, :]
    # three roundings in fp32 (the scales' product, the sum, their product);
    # a product that leaves the normal range is off by half a subnormal step,
    # the scales' times the sum
    tol = 3 * (1 + 2.0 ** -20) * ref.U32 * np.abs(want) + 2.0 ** -149 * (1 + np.abs(acc))
    ref.check(got.cpu().reshape(want.shape), want, tol, f"rows {x.shape[0]} d {x.shape[1]} V {hq.shape[0]}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (5, 8), (1, 512), (9, 520), (4, 2048), (5, 2056), (3, 4096),
                                    (2, 4104), (2, 8192), (2, 8200), (70, 5120), (3, 4099), (300, 64)])
def test_quantize_rows(native, rows, d, dtype):
    x = _rows(rows, d, dtype, rows * 31 + d)
    if rows > 2:
        x[1] = 0.0                                   # a row of zeros
        x[2] = x[2] * 1e-41                          # subnormal numbers, or zeros in bf16's rounding
    q, s = rmd.quantize_rows(x.cuda())
    wq, ws = ref.quantize(x.float().numpy())
    assert q.dtype == torch.int8 and s.dtype == F32 and tuple(s.shape) == (rows,)
    assert np.array_equal(s.cpu().numpy().astype(np.float64), ws)
    assert np.array_equal(q.cpu().numpy().astype(np.float64), wq)


def test_quantize_rows_halves_and_extremes(native):
    """Quotients that end in one half go to the even integer; the type's
    largest values and its smallest do not leave [-127, 127]."""
    x = torch.zeros(6, 16)
    x[0, :6] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5])
    x[1, :3] = torch.tensor([torch.finfo(F32).max, torch.finfo(F32).min, 1.0])
    x[2, :2] = torch.tensor([2.0 ** -149, -2.0 ** -149])
    x[3, :2] = torch.tensor([200 * 2.0 ** -149, -2.0 ** -149])
    x[4, :3] = torch.tensor([float("inf"), 1.0, -2.0])
    x[5, :3] = torch.tensor([float("nan"), 1.0, float("inf")])
    q, s = (t.cpu() for t in rmd.quantize_rows(x.cuda()))
    assert q[0, :6].tolist() == [127, 0, 2, 2, 0, -2]
    assert q[1, :3].tolist() == [127, -127, 0]
    assert s[2] == 0 and not q[2].any()
    wq, ws = ref.quantize(x[3:4].numpy())
    assert s[3].item() == ws[0] and q[3].tolist() == wq[0].astype(int).tolist()
    assert torch.isinf(s[4]) and not q[4].any()
    assert torch.isnan(s[5]) and not q[5].any()


def test_quantize_rows_views_and_outputs(native):
    x = _rows(12, 96, F32, 5).cuda()
    q, s = rmd.quantize_rows(x)
    q2, s2 = rmd.quantize_rows(x.view(3, 4, 96))
    assert torch.equal(q2.view(12, 96), q) and torch.equal(s2.view(12), s)
    qt, st = rmd.quantize_rows(x.t())                # strided: rows of the transpose
    wq, ws = ref.quantize(x.t().cpu().numpy())
    assert np.array_equal(qt.cpu().numpy(), wq) and np.array_equal(st.cpu().numpy(), ws.astype(np.float32))
    off = torch.empty(12 * 96 + 1, device="cuda")[1:].view(12, 96).copy_(x)   # 4-byte aligned
    q3, s3 = rmd.quantize_rows(off)
    assert torch.equal(q3, q) and torch.equal(s3, s)
    buf, sb = torch.full((13, 96), 9, dtype=torch.int8, device="cuda"), torch.full((13,), 9.0, device="cuda")
    out = rmd.quantize_rows(x, out=buf[:12], scale_out=sb[:12])
    assert out[0].data_ptr() == buf.data_ptr() and torch.equal(buf[:12], q) and torch.equal(sb[:12], s)
    assert (buf[12] == 9).all() and sb[12] == 9      # what lies behind stays
    e, es = rmd.quantize_rows(torch.empty(0, 7, device="cuda"))
    assert tuple(e.shape) == (0, 7) and tuple(es.shape) == (0,)
    e, es = rmd.quantize_rows(torch.empty(3, 0, device="cuda"))
    assert tuple(e.shape) == (3, 0) and es.tolist() == [0, 0, 0]


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("rows,V,d", [
    (1, 1, 1), (1, 129, 16), (2, 7, 5), (3, 300, 130), (1, 1000, 5120), (16, 257, 64), (31, 128, 128), (32, 127, 144),
    (33, 515, 272), (64, 256, 256), (65, 1001, 2064), (96, 640, 384), (128, 129, 128), (129, 511, 640), (160, 300, 400),
    (192, 520, 128), (200, 999, 96), (256, 256, 1024), (257, 700, 48), (320, 1030, 176), (330, 257, 1232),
    (513, 383, 80), (700, 130, 16), (2, 9, 4), (33, 200, 12), (70, 131, 516), (150, 1000, 124), (400, 259, 2052), (37, 2003, 2056), (5, 1300, 33), (130, 140, 4099), (1, 40000, 96)])
def test_head_against_64_bits(native, rows, V, d, out):
    x = _rows(rows, d, BF16 if (rows + d) % 2 else F32, rows + V + d)
    hq, hs = _head(V, d, V * 3 + d)
    got = rmd.lm_head_logits_int8(x.cuda(), hq.cuda(), hs.cuda(), out_dtype=out)
    assert got.dtype == out and tuple(got.shape) == (rows, V)
    _check_logits(got, x, hq, hs)


def test_head_largest_sums(native):
    """Every product at 127 * 127: the sum stays below 2^31 up to the largest d."""
    for d in (5120, 131072):
        x = torch.ones(3, d) * torch.tensor([[1.0], [-2.0], [0.0]])
        hq = torch.full((33, d), 127, dtype=torch.int8)
        hq[1] = -127
        hs = torch.full((33,), 0.5)
        got = rmd.lm_head_logits_int8(x.cuda(), hq.cuda(), hs.cuda())
        _check_logits(got, x, hq, hs)


def test_head_rows_that_are_not_numbers(native):
    """A row with an infinity or NaN gives NaN or infinite logits; its
    neighbours keep their values."""
    x = _rows(40, 64, F32, 3)
    hq, hs = _head(100, 64, 4)
    clean = rmd.lm_head_logits_int8(x.cuda(), hq.cuda(), hs.cuda())
    x[7, 5], x[39, 0] = float("nan"), float("inf")
    got = rmd.lm_head_logits_int8(x.cuda(), hq.cuda(), hs.cuda())
    assert not torch.isfinite(got[7]).any() and not torch.isfinite(got[39]).any()
    keep = [i for i in range(40) if i not in (7, 39)]
    assert torch.equal(got[keep], clean[keep])
    x[:] = 0.0
    assert not rmd.lm_head_logits_int8(x.cuda(), hq.cuda(), hs.cuda()).any()


def test_head_views_outputs_and_workspace(native):
    V, d = 700, 256
    x = _rows(24, d, BF16, 1)
    hq, hs = _head(V, d, 2)
    want = rmd.lm_head_logits_int8(x.cuda(), hq.cuda(), hs.cuda())
    _check_logits(want, x, hq, hs)
    ws = rmd.Workspace(4, 6, V, 16, sample=False, int8_hidden=d)
    buf = torch.full((25, V), 5.0, device="cuda")
    got = rmd.lm_head_logits_int8(x.cuda().view(4, 6, d), hq.cuda(), hs.cuda(), out=buf[:24].view(4, 6, V), workspace=ws)
    assert got.data_ptr() == buf.data_ptr() and torch.equal(buf[:24], want) and (buf[24] == 5).all()
    # a strided head, and ones that start at an odd byte and at a word
    wide = torch.zeros(V, d + 32, dtype=torch.int8, device="cuda")
    wide[:, :d] = hq.cuda()
    assert torch.equal(rmd.lm_head_logits_int8(x.cuda(), wide[:, :d], hs.cuda()), want)
    for off in (1, 4):
        odd = torch.zeros(V * d + off, dtype=torch.int8, device="cuda")
        odd[off:] = hq.cuda().view(-1)
        assert torch.equal(rmd.lm_head_logits_int8(x.cuda(), odd[off:].view(V, d), hs.cuda()), want)
    # an output that starts at an odd element
    flat = torch.empty(24 * V + 1, device="cuda", dtype=BF16)
    got = rmd.lm_head_logits_int8(x.cuda(), hq.cuda(), hs.cuda(), out=flat[1:].view(24, V))
    assert torch.equal(got, want.to(BF16))
    assert tuple(rmd.lm_head_logits_int8(x[:0].cuda(), hq.cuda(), hs.cuda()).shape) == (0, V)


def test_head_too_small_a_workspace_is_refused(native):
    ws = rmd.Workspace(1, 1, 64, 16, sample=False)
    hq, hs = _head(64, 64, 1)
    from rank_markov_draft_amd import _lib
    with pytest.raises(_lib.DsparkError, match="WORKSPACE"):
        rmd.lm_head_logits_int8(torch.zeros(4096, 64, device="cuda"), hq.cuda(), hs.cuda(), workspace=ws)


def test_head_is_the_same_twice_and_on_another_stream(native):
    x, (hq, hs) = _rows(70, 512, BF16, 8).cuda(), _head(5000, 512, 9)
    hq, hs = hq.cuda(), hs.cuda()
    want = rmd.lm_head_logits_int8(x, hq, hs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = rmd.lm_head_logits_int8(x, hq, hs)
    b = rmd.lm_head_logits_int8(x, hq, hs)           # at the same time, its own workspace
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


def test_head_past_31_bits(native):
    """A head of over 2^31 bytes and logits of over 2^31 bytes."""
    V, d, rows = 132000, 16512, 4200
    g = torch.Generator(device="cuda").manual_seed(5)
    hq = torch.randint(-127, 128, (V, d), device="cuda", generator=g, dtype=torch.int8)
    hs = torch.rand(V, device="cuda", generator=g) * 1e-3
    x = torch.randn(rows, d, device="cuda", generator=g).to(BF16)
    assert V * d > 2 ** 31 and rows * V * 4 > 2 ** 31
    got = rmd.lm_head_logits_int8(x, hq, hs)
    r = torch.tensor([0, 1, 255, 256, 2100, rows - 1])
    c = torch.tensor([0, 7, 65535, 130060, 131000, V - 2, V - 1])
    _check_logits(got[r][:, c], x[r].cpu(), hq[c].cpu(), hs[c].cpu())
    one = rmd.lm_head_logits_int8(x[-1:], hq, hs)    # the single token form on the same head
    assert torch.equal(one[0], got[-1])


def test_head_in_a_graph(native):
    V, d = 3000, 320
    x, (hq, hs) = torch.zeros(10, d, device="cuda", dtype=BF16), _head(V, d, 3)
    hq, hs = hq.cuda(), hs.cuda()
    ws = rmd.Workspace(10, 1, V, 16, sample=False, int8_hidden=d)
    out = torch.empty(10, V, device="cuda")
    rmd.lm_head_logits_int8(x, hq, hs, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rmd.lm_head_logits_int8(x, hq, hs, out=out, workspace=ws)
    for k in range(4):
        x.copy_(_rows(10, d, BF16, 50 + k))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        eager = rmd.lm_head_logits_int8(x, hq, hs)
        assert torch.equal(got, eager) and got.any()


def test_int8_head_feeds_the_draft(native):
    """As a server runs it: the head's rows quantised once, base logits by the
    8-bit head, then the left-to-right draft under the request's rules."""
    B, M, V, d, r = 3, 4, 1000, 256, 16
    g = torch.Generator().manual_seed(1)
    lm = (torch.randn(V, d, generator=g) * 0.1).to(BF16).cuda()
    hidden = torch.randn(B, M, d, generator=g).to(BF16).cuda()
    w1, w2 = ((torch.randn(V, r, generator=g) * 0.02).to(BF16).cuda() for _ in range(2))
    first = torch.tensor([1, 2, 3], device="cuda")
    hq, hs = rmd.quantize_rows(lm)
    base = rmd.lm_head_logits_int8(hidden, hq, hs)
    assert tuple(base.shape) == (B, M, V)
    # half a step of each factor: |x - s q| <= s / 2 per element, on both sides
    full = hidden.float() @ lm.float().t()
    xs = rmd.quantize_rows(hidden)[1]
    bound = (xs[..., None] / 2) * lm.float().abs().sum(-1) + (hs / 2) * (hidden.float().abs() + xs[..., None] / 2).sum(-1, keepdim=True)
    assert ((base - full).abs() <= bound * 1.001 + 1e-4).all()
    allowed = np.zeros((B, V), bool)
    allowed[:, ::7] = True
    mask = torch.from_numpy(ref.pack_mask(allowed)).cuda()
    rep = torch.full((B,), 1.2, device="cuda")
    tok, proc = rmd.sample_block_tokens_processed(base, first, w1, w2, 0.0, history=first[:, None], repetition_penalty=rep,
                                                  token_mask=mask)
    assert (tok % 7 == 0).all()
    assert torch.equal(proc.cpu().argmax(-1), tok.cpu())


@pytest.mark.parametrize("d", [144, 148, 151])
@pytest.mark.parametrize("rows,V", [(5, 200), (40, 300), (64, 70000), (65, 70000), (192, 70001), (250, 70000), (320, 70100),
                                    (512, 33000), (321, 70000)])
def test_every_tile_form(native, rows, V, d):
    """Sizes on both sides of the rule that picks the tile, heads read straight
    into LDS by pieces (d a multiple of 16) or words (of 4) and through
    registers; several tiles a workgroup, and the last of them partial."""
    x = _rows(rows, d, BF16, rows + d).cuda()
    hq, hs = (t.cuda() for t in _head(V, d, V))
    for out in (F32, BF16):
        got = rmd.lm_head_logits_int8(x, hq, hs, out_dtype=out)
        q, s = rmd.quantize_rows(x)
        # sums of 151 products of 127 * 127 are whole numbers below 2^24: exact in fp32
        acc = q.float() @ hq.float().t()
        want = ((s[:, None] * hs[None, :]) * acc).to(out)
        assert torch.equal(got, want)
