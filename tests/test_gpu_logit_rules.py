"""Penalties, biases and grammar masks on the GPU against 64 bits; the
gradient against the formula and against differences; the left-to-right draft
row by row."""
import numpy as np
import pytest
import torch

import rank_markov_draft_amd as rmd
from oracle import oracle as orc
from tests import parity
from tests import rules_reference as ref
from tests.gpu_util import from_dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


class Case:
    """Host inputs of a call and its rules; ``kw(M)`` the keyword arguments on the GPU."""

    def __init__(self, B, M, V, L, dtype, mask="each", bias="row", seed=0, penalties=True, bias_dtype=F32):
        g = np.random.default_rng(seed + 17 * B + 3 * M + V + L)
        self.B, self.M, self.V, self.dtype = B, M, V, dtype
        self.logits = torch.from_numpy(g.standard_normal((B, M, V)).astype(np.float32) * 3).to(dtype)
        hot = max(1, V // 5)  # repeats
        self.history = g.integers(0, hot, (B, L)) if L >= 0 else None
        self.lengths = g.integers(0, L + 1, B) if L >= 0 else None
        self.prompt = None
        if L >= 0:
            self.lengths[0] = L
            if B > 1:
                self.lengths[1] = 0
            self.prompt = (self.lengths * g.random(B)).astype(np.int64)
            for b in range(B):
                self.history[b, self.lengths[b]:] = -7   # not read
        self.ids = g.integers(0, hot, (B, M))
        self.rep = (1.0 + g.random(B)).astype(np.float32) if penalties else None
        self.freq = g.random(B).astype(np.float32) if penalties else None
        self.pres = g.random(B).astype(np.float32) if penalties else None
        if penalties and B > 2:
            self.rep[2], self.freq[2] = 0.7, -0.3        # repetition encouraged
        self.bias = None
        if bias != "none":
            self.bias = torch.from_numpy(g.standard_normal((V,) if bias == "shared" else (B, V)).astype(np.float32)).to(bias_dtype)
        self.allowed = None
        if mask != "none":
            shape = {"each": (B, M, V), "row": (B, 1, V), "shared": (1, 1, V)}[mask]
            self.allowed = g.random(shape) < 0.6
            self.allowed[-1, -1] = False                 # nothing is left
        self.mask = None if self.allowed is None else ref.pack_mask(self.allowed)
        if self.mask is not None and V % 32:             # bits past the vocabulary mean nothing
            self.mask = (self.mask.view(np.uint32) | np.where(np.arange(self.mask.shape[-1]) == self.mask.shape[-1] - 1,
                                                              np.uint32(0xFFFFFFFF) << np.uint32(V % 32), 0).astype(np.uint32)).view(np.int32)

    def kw(self, backward=False):
        dev = lambda a: None if a is None else (torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a).cuda()  # noqa: E731
        kw = dict(history=dev(self.history), lengths=dev(self.lengths), prompt_lengths=dev(self.prompt),
                  repetition_penalty=dev(self.rep), token_mask=dev(self.mask))
        if not backward:
            kw.update(frequency_penalty=dev(self.freq), presence_penalty=dev(self.pres), logit_bias=dev(self.bias))
        return kw

    def allowed_row(self, b, k):
        if self.allowed is None:
            return None
        a = self.allowed
        return a[b if a.shape[0] > 1 else 0, k if a.shape[1] > 1 else 0]

    def row(self, x, b, k, extra):
        n = lambda a: None if a is None else float(a[b])  # noqa: E731
        count, seen = ref.counts(self.history, self.lengths, self.prompt, extra, b, self.V)
        bias = None
        if self.bias is not None:
            bias = (self.bias if self.bias.dim() == 1 else self.bias[b]).double().numpy()
        return ref.rules_row(x, count, seen, n(self.rep), n(self.freq), n(self.pres), bias, self.allowed_row(b, k))

    def want(self, ids=True):
        out = [self.row(self.logits[b, k].double().numpy(), b, k, self.ids[b, 1:k + 1] if ids else ())
               for b in range(self.B) for k in range(self.M)]
        return np.stack([o[0] for o in out]), np.stack([o[1] for o in out])


SIZES = [(1, 1, 1, 0), (1, 1, 7, 1), (1, 1, 2048, 50), (2, 3, 2051, 5), (3, 2, 4096, 300), (5, 4, 1001, 64),
         (4, 5, 8200, 2100), (1, 8, 16385, 9), (40, 2, 8191, 33), (130, 1, 8193, 20), (3, 3, 33, 2049), (600, 1, 40, 3),
         (1, 67, 301, 20), (2, 33, 97, 4), (3, 300, 40, 5), (1, 515, 65, 3), (1100, 17, 50, 6)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,M,V,L", SIZES)
def test_rules_against_64_bits(native, B, M, V, L, dtype):
    c = Case(B, M, V, L, dtype, mask=("each", "row", "shared")[(B + V) % 3], bias=("row", "shared")[(M + V) % 2],
             bias_dtype=(F32, BF16)[V % 2])
    ids = torch.from_numpy(c.ids).cuda()
    got = rmd.process_block_logits(c.logits.cuda(), token_ids=ids, **c.kw())
    assert got.dtype == dtype and tuple(got.shape) == (B, M, V)
    want, tol = c.want()
    ref.check(got.reshape(B * M, V), want, tol, f"{B}x{M}x{V} L {L}")
    # in place, and without the block's own tokens
    x = c.logits.cuda()
    assert rmd.process_block_logits(x, token_ids=ids, out=x, **c.kw()) is x and torch.equal(x, got)
    alone = rmd.process_block_logits(c.logits.cuda(), **c.kw())
    want, tol = c.want(ids=False)
    ref.check(alone.reshape(B * M, V), want, tol, "without token_ids")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("on", ["rep", "freq", "pres", "bias", "mask", "none", "ids"])
def test_each_rule_by_itself(native, on, dtype):
    c = Case(3, 4, 777, 40, dtype)
    keep = {"rep": "rep", "freq": "freq", "pres": "pres", "bias": "bias", "mask": "allowed", "ids": "rep"}.get(on)
    for name in ("rep", "freq", "pres", "bias", "allowed"):
        if name != keep:
            setattr(c, name, None)
    if on != "mask":
        c.mask = None
    if on == "ids":  # the block's tokens without any history
        c.history = c.lengths = c.prompt = None
    got = rmd.process_block_logits(c.logits.cuda(), token_ids=torch.from_numpy(c.ids).cuda(), **c.kw())
    want, tol = c.want()
    ref.check(got.reshape(12, 777), want, tol, on)
    if on == "none":
        assert torch.equal(got.cpu(), c.logits)


def test_masked_places_and_infinities(native):
    """Infinities, NaN and the type's lowest value, masked and not, seen and not."""
    for dtype in (F32, BF16):
        V = 64
        vals = torch.tensor([float("inf"), -float("inf"), float("nan"), torch.finfo(dtype).min, torch.finfo(dtype).max, 0.0, -0.0, 1.0])
        x = vals.repeat(V // 8).to(dtype).view(1, 1, V)
        c = Case(1, 1, V, 0, dtype, mask="none", bias="none")
        c.logits = x
        c.history, c.lengths, c.prompt = np.arange(32)[None], np.array([32]), np.array([16])
        c.rep, c.freq, c.pres = np.array([1.5], np.float32), np.array([0.25], np.float32), np.array([0.5], np.float32)
        c.allowed = (np.arange(V) % 16 < 8)[None, None]
        c.mask = ref.pack_mask(c.allowed)
        got = rmd.process_block_logits(x.cuda(), **c.kw())
        want, tol = c.want(ids=False)
        ref.check(got.reshape(1, V), want, tol, str(dtype))
        assert (got[0, 0, ~torch.from_numpy(c.allowed[0, 0]).cuda()] == -float("inf")).all()
        g = torch.full_like(x, float("nan"))
        back = rmd.process_block_logits_backward(g.cuda(), x.cuda(), **c.kw(backward=True)).cpu()
        assert not back[0, 0, ~torch.from_numpy(c.allowed[0, 0])].any()   # zero, whatever stood there


def test_lengths_out_of_range_and_foreign_ids(native):
    V = 300
    c = Case(3, 1, V, 12, F32, mask="none", bias="none")
    c.history[:] = np.random.default_rng(3).integers(0, V, (3, 12))
    c.history[0, 3:6] = [-1, V, 2 ** 40]
    c.history[1, 0] = -2 ** 62
    c.lengths[:] = [12, 99, -5]                      # clamped to 12, 12 and 0
    c.prompt[:] = [-3, 5, 50]
    got = rmd.process_block_logits(c.logits.cuda(), **c.kw())
    want, tol = c.want(ids=False)
    ref.check(got.reshape(3, V), want, tol, "clamped lengths")
    c.ids[:] = -1
    c.M = 1
    assert torch.equal(rmd.process_block_logits(c.logits.cuda(), token_ids=torch.from_numpy(c.ids).cuda(), **c.kw()), got)


def test_views_strides_and_alignment(native):
    B, M, V, L = 3, 2, 515, 20
    c = Case(B, M, V, L, BF16)
    ids = torch.from_numpy(c.ids).cuda()
    want = rmd.process_block_logits(c.logits.cuda(), token_ids=ids, **c.kw())
    kw = c.kw()
    # logits at odd elements, an output that differs in alignment, a strided batch
    for off_in, off_out in ((0, 1), (1, 0), (1, 1), (3, 5), (7, 7)):
        x = torch.empty(B * M * V + off_in, device="cuda", dtype=BF16)[off_in:].view(B, M, V).copy_(c.logits)
        full = torch.full((B * M * V + off_out + 3,), 9.0, device="cuda", dtype=BF16)
        o = full[off_out:off_out + B * M * V].view(B, M, V)
        assert torch.equal(rmd.process_block_logits(x, token_ids=ids, out=o, **kw), want)
        assert (full[:off_out] == 9).all() and (full[off_out + B * M * V:] == 9).all()
        g = rmd.process_block_logits_backward(x, c.logits.cuda(), token_ids=ids, out=o, **c.kw(backward=True))
        assert torch.equal(g, rmd.process_block_logits_backward(c.logits.cuda(), c.logits.cuda(), token_ids=ids, **c.kw(backward=True)))
    x = c.logits.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(rmd.process_block_logits(x, token_ids=ids, **kw), want)
    # history inside a larger buffer, int32 ids, a mask with strides, expanded
    big = torch.full((B, 2 * L), 3, device="cuda")
    big[:, :L] = kw["history"]
    kw2 = dict(kw, history=big[:, :L], token_mask=kw["token_mask"].transpose(0, 1).contiguous().transpose(0, 1))
    assert torch.equal(rmd.process_block_logits(x, token_ids=ids.int(), **kw2), want)
    kw2["history"] = kw["history"].int()
    assert torch.equal(rmd.process_block_logits(x, token_ids=ids, **kw2), want)
    m = kw["token_mask"][:1, :1]
    a = rmd.process_block_logits(x, token_ids=ids, **dict(kw, token_mask=m))
    b = rmd.process_block_logits(x, token_ids=ids, **dict(kw, token_mask=m.expand(B, M, -1)))
    d = rmd.process_block_logits(x, token_ids=ids, **dict(kw, token_mask=m.expand(B, M, -1).contiguous()))
    assert torch.equal(a, b) and torch.equal(a, d)


def test_long_history_counts(native):
    """A history of one token, and of more ids than a tile has columns."""
    V, L = 3000, 70001
    c = Case(2, 1, V, 0, F32, mask="none", bias="none")
    c.history = np.random.default_rng(1).integers(0, V, (2, L))
    c.history[0, :] = 5
    c.lengths, c.prompt = np.array([L, L - 1]), np.array([1, L // 2])
    got = rmd.process_block_logits(c.logits.cuda(), **c.kw())
    want, tol = c.want(ids=False)
    ref.check(got.reshape(2, V), want, tol, "long history")


def test_empty_calls(native):
    for shape in ((0, 3, 8), (2, 0, 8), (2, 3, 0)):
        x = torch.empty(shape, device="cuda")
        assert rmd.process_block_logits(x).shape == x.shape
        assert rmd.process_block_logits_backward(x, x).shape == x.shape
    c = Case(2, 1, 50, 0, F32, mask="none", bias="none")     # a history without a column
    got = rmd.process_block_logits(c.logits.cuda(), **c.kw())
    assert torch.equal(got.cpu(), c.logits)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,M,V,L", SIZES)
def test_gradient_against_the_formula(native, B, M, V, L, dtype):
    c = Case(B, M, V, L, dtype, mask=("each", "row", "shared", "none")[(B + V) % 4])
    g = torch.from_numpy(np.random.default_rng(5).standard_normal((B, M, V)).astype(np.float32)).to(dtype)
    if V > 4:
        c.logits[:, :, 3] = 0.0                     # the corner: the slope of the lower side
        c.logits[0, 0, 2] = float("nan")
    ids = torch.from_numpy(c.ids).cuda()
    got = rmd.process_block_logits_backward(g.cuda(), c.logits.cuda(), token_ids=ids, **c.kw(backward=True))
    want = np.empty((B * M, V))
    tol = np.empty_like(want)
    for b in range(B):
        for k in range(M):
            _, seen = ref.counts(c.history, c.lengths, c.prompt, c.ids[b, 1:k + 1], b, V)
            x = c.logits[b, k].double().numpy()
            w = g[b, k].double().numpy() * np.where(seen, np.where(x > 0, 1.0 / float(c.rep[b]), float(c.rep[b])), 1.0)
            a = c.allowed_row(b, k)
            want[b * M + k] = w if a is None else np.where(a, w, 0.0)
            tol[b * M + k] = np.where(seen, ref.U32 * np.abs(w), 0.0)
    ref.check(got.reshape(B * M, V), want, tol, "gradient")
    gd = g.cuda()
    assert rmd.process_block_logits_backward(gd, c.logits.cuda(), token_ids=ids, out=gd, **c.kw(backward=True)) is gd
    assert torch.equal(gd, got)


def test_gradient_against_differences_and_through_the_head(native):
    """loss = sum of G times the processed corrected logits: the rules'
    gradient, then the head's, against central differences of the plain form
    in 64 bits (the loss is piecewise linear in the base logits, and in W2 for
    fixed W1)."""
    B, M, V, r = 2, 3, 40, 8
    c = Case(B, M, V, 12, F32, mask="none", bias="row")
    rng = np.random.default_rng(2)
    c.allowed = rng.random((B, M, V)) < 0.8
    c.mask = ref.pack_mask(c.allowed)
    G = np.where(c.allowed, rng.standard_normal((B, M, V)), 0.0).astype(np.float32)
    w1, w2 = (rng.standard_normal((V, r)).astype(np.float32) * 0.3 for _ in range(2))
    base, ids = c.logits.numpy().astype(np.float64), c.ids

    def corrected(bs, w):
        return bs + np.einsum("bkr,vr->bkv", w1.astype(np.float64)[ids], w)

    def loss(bs, w):
        x, s = corrected(bs, w), 0.0
        for b in range(B):
            for k in range(M):
                y, _ = c.row(x[b, k], b, k, ids[b, 1:k + 1])
                s += float((np.where(c.allowed[b, k], y, 0.0) * G[b, k]).sum())
        return s

    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    corr = rmd.apply_block_logits(c.logits.cuda(), t(ids), t(w1), t(w2))
    proc = rmd.process_block_logits(corr, token_ids=t(ids), **c.kw())
    assert torch.isfinite(proc[t(c.allowed)]).all()
    dx = rmd.process_block_logits_backward(t(G), corr, token_ids=t(ids), **c.kw(backward=True))
    _, dw2 = rmd.apply_block_logits_backward(dx, t(ids), t(w1), t(w2))
    x0, h = corrected(base, w2.astype(np.float64)), 2.0 ** -20
    for b, k, v in [(0, 0, 1), (0, 2, 5), (1, 1, 0), (1, 2, 39), (1, 0, 7), (0, 1, 3)]:
        if abs(x0[b, k, v]) < 1e-3:
            continue
        e = np.zeros_like(base)
        e[b, k, v] = h
        d = (loss(base + e, w2.astype(np.float64)) - loss(base - e, w2.astype(np.float64))) / (2 * h)
        # differences of sums of 240 terms of a few units, in 64 bits over 2 h = 2^-19, and one rounding
        assert abs(dx[b, k, v].item() - d) <= 240 * 16 * 2.0 ** -53 * 2 ** 19 + 2.0 ** -24 * abs(d)
    for v, j in [(0, 0), (3, 5), (17, 2), (39, 7)]:
        if np.abs(x0[:, :, v]).min() < 1e-3:
            continue
        e = np.zeros((V, r))
        e[v, j] = h
        d = (loss(base, w2 + e) - loss(base, w2 - e)) / (2 * h)
        scale = np.abs(dx[:, :, v].cpu().numpy()).sum() * np.abs(w1).max()
        assert abs(dw2[v, j].item() - d) <= 240 * 16 * 2.0 ** -53 * 2 ** 19 + 10 * 2.0 ** -24 * scale


# ------------------------------------------------------------ left to right
def _draft_case(B, M, V, L, r, ldt, wdt, seed=0, **kw):
    c = Case(B, M, V, L, ldt, seed=seed, **kw)
    g = np.random.default_rng(seed + 99)
    c.first = g.integers(0, V, B)
    c.w1, c.w2 = (torch.from_numpy(g.standard_normal((V, r)).astype(np.float32) * 0.2).to(wdt) for _ in range(2))
    return c


def _draft(c, T=0.0, **kw):
    return rmd.sample_block_tokens_processed(c.logits.cuda(), torch.from_numpy(c.first).cuda(), c.w1.cuda(), c.w2.cuda(), T,
                                             **c.kw(), **kw)


def _check_draft(c, tokens, rows, T=0.0, seed=0, pos=0, bat=0):
    """Each processed row against the definition given the tokens drawn before
    it, and each token as the selection on the GPU's own row."""
    tok = tokens.cpu().numpy()
    V, r, ldt, wdt = c.V, c.w1.shape[1], c.dtype, c.w1.dtype
    w1, w2 = c.w1.double().numpy(), c.w2.double().numpy()
    for b in range(c.B):
        for k in range(c.M):
            x = int(c.first[b]) if k == 0 else int(tok[b, k - 1])
            e = w1[x] if 0 <= x < V else np.zeros(r)
            bias = w2 @ e
            # fp32 accumulation in any order, the Linear's rounding, the cast
            # to the logits' type, then the sum's rounding
            tb = 2 * r * ref.U32 * (np.abs(w2) @ np.abs(e))
            tb = tb + ref.HALF_STEP[wdt] * (np.abs(bias) + tb)
            if ldt != wdt:
                tb = tb + ref.HALF_STEP[ldt] * (np.abs(bias) + tb)
            s = c.logits[b, k].double().numpy() + bias
            tc = tb + ref.U32 * (np.abs(s) + tb)
            tc = tc + ref.HALF_STEP[ldt] * (np.abs(s) + tc)
            want, tol = c.row(s, b, k, tok[b, :k])
            steep = 1.0 if c.rep is None else max(1.0, float(c.rep[b]), 1.0 / float(c.rep[b]))
            got = rows[b, k]
            ref.check(got, want, (tol + tc * steep) * (1 + 2.0 ** -8), f"row {b} {k}")
            if not (got > -float("inf")).any() and not torch.isnan(got).any():
                assert tok[b, k] == -1
                continue
            own = from_dev(got.reshape(1, V))
            parity.check_tokens(tok[b:b + 1, k], own, None, T, seed, [bat + b], [pos + k])


@pytest.mark.parametrize("T", [0.0, 0.7])
@pytest.mark.parametrize("B,M,V,L,r,ldt,wdt", [
    (1, 1, 1, 1, 1, F32, F32), (1, 1, 5000, 10, 16, BF16, BF16), (3, 4, 1000, 40, 16, BF16, BF16),
    (2, 5, 4104, 100, 256, BF16, BF16), (4, 3, 1001, 20, 10, BF16, BF16), (3, 3, 2000, 30, 64, F32, BF16),
    (2, 3, 999, 30, 64, F32, F32), (2, 2, 1000, 5, 12, F32, F32), (3, 2, 520, 8, 40, BF16, F32),
    (2, 2, 9000, 64, 512, BF16, BF16), (33, 2, 264, 7, 8, BF16, BF16)])
def test_draft_under_rules(native, B, M, V, L, r, ldt, wdt, T):
    c = _draft_case(B, M, V, L, r, ldt, wdt, mask=("each", "row", "none")[(B + M) % 3], bias=("row", "shared", "none")[V % 3])
    tok, rows = _draft(c, T, seed=77, position_offset=2, batch_offset=5)
    assert tok.dtype == torch.int64 and tuple(tok.shape) == (B, M) and rows.dtype == ldt
    _check_draft(c, tok, rows, T, 77, 2, 5)


@pytest.mark.parametrize("T", [0.0, 0.9])
@pytest.mark.parametrize("B,M,V,L,r,ldt,wdt", [
    (4, 4, 777, 30, 33, BF16, BF16), (1, 3, 2050, 20, 1, F32, F32), (2, 3, 515, 9, 130, F32, F32), (4, 3, 1030, 40, 1000, F32, BF16),
    (3, 3, 65, 9, 258, BF16, F32), (4, 5, 3, 6, 7, F32, F32), (5, 3, 1001, 20, 10, BF16, BF16), (7, 3, 999, 30, 64, F32, F32),
    (16, 2, 2000, 30, 300, F32, BF16), (9, 2, 520, 8, 40, BF16, F32), (12, 4, 97, 5, 13, F32, F32), (5, 2, 9000, 64, 512, BF16, BF16),
    (20, 3, 265, 7, 300, F32, F32), (32, 2, 1999, 20, 72, BF16, F32), (40, 3, 1001, 20, 130, F32, F32), (70, 2, 130, 9, 24, BF16, F32)])
def test_draft_of_more_sizes_under_rules(native, B, M, V, L, r, ldt, wdt, T):
    c = _draft_case(B, M, V, L, r, ldt, wdt, mask=("each", "row", "none")[(B + M) % 3], bias=("row", "shared", "none")[V % 3])
    tokens, rows = _draft(c, T=T, seed=5, position_offset=2, batch_offset=1)
    _check_draft(c, tokens, rows, T=T, seed=5, pos=2, bat=1)


@pytest.mark.parametrize("T", [0.0, 0.8])
@pytest.mark.parametrize("B,M,V,L,r,ldt,wdt", [
    (16, 2, 33001, 20, 10, BF16, BF16), (8, 2, 66001, 30, 16, F32, F32), (13, 2, 40002, 9, 40, F32, BF16), (16, 2, 33000, 5, 13, BF16, F32),
    (32, 2, 16510, 20, 72, BF16, F32), (20, 2, 26305, 9, 33, F32, F32), (32, 2, 16640, 9, 520, F32, BF16), (40, 2, 13201, 7, 24, BF16, BF16),
    (64, 2, 8501, 9, 130, F32, BF16), (70, 3, 8001, 5, 7, F32, F32), (33, 2, 15003, 30, 300, BF16, F32),
    (64, 2, 70001, 9, 8, BF16, BF16), (300, 2, 16385, 5, 16, F32, BF16), (130, 2, 16400, 5, 9, BF16, F32), (100, 2, 33001, 5, 8, F32, F32)])
def test_draft_of_many_columns_and_rows(native, B, M, V, L, r, ldt, wdt, T):
    """Sizes that more than fill the device four rows a workgroup: they run by row tiles."""
    assert -(-V // 256) * -(-B // 4) > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    c = _draft_case(B, M, V, L, r, ldt, wdt, mask=("each", "row", "none")[(B + M) % 3], bias=("row", "shared", "none")[V % 3])
    tokens, rows = _draft(c, T=T, seed=6, position_offset=1, batch_offset=3)
    _check_draft(c, tokens, rows, T=T, seed=6, pos=1, bat=3)


def test_draft_without_rules_is_the_plain_draft(native):
    c = _draft_case(4, 5, 4096, -1, 64, BF16, BF16, mask="none", bias="none", penalties=False)
    for T in (0.0, 0.9):
        tok, rows = _draft(c, T, seed=3)
        t2, r2 = rmd.sample_block_tokens(c.logits.cuda(), torch.from_numpy(c.first).cuda(), c.w1.cuda(), c.w2.cuda(), T, seed=3)
        _check_draft(c, tok, rows, T, 3)
        # the plain draft sums the bias on another kernel: a flip of the last
        # bit is allowed by _check_draft, so tokens may differ only where rows do
        same = (rows == r2).all(-1)
        first_change = (tok != t2)
        assert not (first_change[:, 0] & same[:, 0]).any()


def test_draft_counts_what_it_draws(native):
    """A confident token is drawn once under a large presence penalty, and its
    own history is the draft's: five positions give five tokens."""
    B, M, V = 2, 5, 300
    c = _draft_case(B, M, V, -1, 8, F32, F32, mask="none", bias="none", penalties=False)
    c.logits.zero_()
    c.logits[:, :, :6] = torch.tensor([60.0, 50, 40, 30, 20, 10])
    c.w1.zero_()
    c.pres = np.full(B, 100.0, np.float32)
    tok, rows = _draft(c)
    assert tok.tolist() == [[0, 1, 2, 3, 4]] * B
    _check_draft(c, tok, rows)
    c.pres, c.rep = None, np.full(B, 10.0, np.float32)
    assert _draft(c)[0].tolist() == [[0, 1, 2, 3, 4]] * B
    c.rep, c.freq = None, np.full(B, 15.0, np.float32)
    tok, rows = _draft(c)
    _check_draft(c, tok, rows)
    assert tok.tolist() == [[0, 1, 0, 2, 1]] * B


def test_draft_rows_with_nothing_left(native):
    c = _draft_case(3, 3, 200, 10, 8, BF16, BF16, mask="each", bias="none")
    c.allowed[1, 1] = False
    c.mask = ref.pack_mask(c.allowed)
    ws = rmd.Workspace(3, 3, 200, 8, sample=True, processed=True)
    tok, rows = _draft(c, workspace=ws)
    assert tok[1, 1] == -1 and tok[2, 2] == -1 and (tok[0] >= 0).all() and tok[1, 2] >= 0
    assert (rows[1, 1] == -float("inf")).all()
    _check_draft(c, tok, rows)
    tok, rows = _draft(c, 0.5, seed=4, workspace=ws)
    assert tok[1, 1] == -1 and tok[2, 2] == -1
    _check_draft(c, tok, rows, 0.5, 4)


def test_draft_one_token_at_a_time(native):
    """M calls of one position, the history grown by the tokens drawn, give the
    whole draft (a grammar whose mask follows the tokens is served so)."""
    for ldt, wdt, V in ((F32, F32, 501), (BF16, BF16, 512)):
        for T in (0.0, 0.8):
            c = _draft_case(3, 4, V, 12, 16, ldt, wdt, mask="each")
            tok, rows = _draft(c, T, seed=5)
            kw = c.kw()
            buf = torch.full((3, 20), -1, device="cuda")
            buf[:, :12] = kw.pop("history")
            length = kw.pop("lengths")
            mask = kw.pop("token_mask")
            prev = torch.from_numpy(c.first).cuda()
            for k in range(4):
                t, rk = rmd.sample_block_tokens_processed(c.logits[:, k:k + 1].cuda(), prev, c.w1.cuda(), c.w2.cuda(), T, seed=5,
                                                          position_offset=k, history=buf, lengths=length,
                                                          token_mask=mask[:, k:k + 1], **kw)
                assert torch.equal(t[:, 0], tok[:, k]) and torch.equal(rk[:, 0], rows[:, k])
                prev = t[:, 0]
                buf.scatter_(1, length[:, None], t)
                length = length + 1


def test_draft_bad_predecessors_and_shared_workspace(native):
    c = _draft_case(2, 2, 128, 4, 8, BF16, BF16, mask="none")
    c.first[:] = [-1, 128]
    ws = rmd.Workspace(2, 2, 128, 8, sample=True, processed=True)
    tok, rows = _draft(c, workspace=ws)
    _check_draft(c, tok, rows)
    assert rmd.read_device_error(ws) == 2
    # the plain draft and the teacher-forced calls run on the same workspace
    c.first[:] = [0, 1]
    dev = (c.logits.cuda(), torch.from_numpy(c.first).cuda(), c.w1.cuda(), c.w2.cuda())
    want = rmd.sample_block_tokens(*dev)
    a = rmd.sample_block_tokens(*dev, workspace=ws)
    again = _draft(c, workspace=ws)
    fresh = _draft(c)
    b = rmd.sample_block_tokens(*dev, workspace=ws)
    for t in (a, b):
        assert torch.equal(t[0], want[0]) and torch.equal(t[1], want[1])
    assert torch.equal(again[0], fresh[0]) and torch.equal(again[1], fresh[1])


def test_two_drafts_at_once_and_outputs(native):
    c = _draft_case(6, 3, 3000, 50, 32, BF16, BF16)
    want = _draft(c, 0.6, seed=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = _draft(c, 0.6, seed=9)
    tok, rows = torch.full((7, 3), 5, device="cuda"), torch.full((7, 3, 3000), 5.0, device="cuda", dtype=BF16)
    b = _draft(c, 0.6, seed=9, tokens_out=tok[:6], logits_out=rows[:6])
    torch.cuda.synchronize()
    for t in (a, b):
        assert torch.equal(t[0], want[0]) and torch.equal(t[1], want[1])
    assert b[0].data_ptr() == tok.data_ptr() and (tok[6] == 5).all() and (rows[6] == 5).all()


def test_rules_and_draft_in_a_graph(native):
    """Captured once, replayed on new logits, lengths and masks."""
    B, M, V, L = 4, 3, 2050, 64
    c = _draft_case(B, M, V, L, 16, BF16, BF16, mask="each")
    kw = c.kw()
    x, ids = c.logits.cuda(), torch.from_numpy(c.ids).cuda()
    first, w1, w2 = torch.from_numpy(c.first).cuda(), c.w1.cuda(), c.w2.cuda()
    ws = rmd.Workspace(B, M, V, 16, sample=True, processed=True)
    out, tok, rows = torch.empty_like(x), torch.empty(B, M, dtype=torch.int64, device="cuda"), torch.empty_like(x)

    def step(**more):
        rmd.process_block_logits(x, token_ids=ids, out=out, **kw)
        rmd.sample_block_tokens_processed(x, first, w1, w2, 0.0, tokens_out=tok, logits_out=rows, workspace=ws, **kw)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator(device="cuda").manual_seed(1)
    for k in range(4):
        x.copy_(torch.randn(x.shape, device="cuda", generator=g) * 3)
        kw["lengths"].copy_(torch.randint(0, L + 1, (B,), device="cuda", generator=g))
        kw["history"].copy_(torch.randint(0, V, (B, L), device="cuda", generator=g))
        kw["token_mask"].bitwise_not_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), tok.clone(), rows.clone()
        eager = rmd.process_block_logits(x, token_ids=ids, **kw)
        et, er = rmd.sample_block_tokens_processed(x, first, w1, w2, 0.0, **kw)
        assert torch.equal(got[0], eager) and torch.equal(got[1], et) and torch.equal(got[2], er)


@pytest.mark.parametrize("B", [3, 20])
def test_two_graphs_share_a_workspace(native, B):
    """The 8-bit head and a greedy draft in the chain as one graph, a draft by
    steps (no penalty: no table) as another, replayed in turn on one workspace
    with eager calls between."""
    M, V, L, r, d = 4, 2048, 64, 16, 192
    c = _draft_case(B, M, V, L, r, BF16, BF16, mask="each", bias="shared")
    kw, first, w1, w2 = c.kw(), torch.from_numpy(c.first).cuda(), c.w1.cuda(), c.w2.cuda()
    plain = dict(token_mask=kw["token_mask"], logit_bias=kw["logit_bias"])
    g = torch.Generator(device="cuda").manual_seed(B)
    hidden = torch.randn(B, M, d, device="cuda", generator=g).to(BF16)
    hq, hs = rmd.quantize_rows(torch.randn(V, d, device="cuda", generator=g) * 0.2)
    ws = rmd.Workspace(B, M, V, r, sample=True, processed=True, int8_hidden=d)

    def one(h, **more):
        base = rmd.lm_head_logits_int8(h, hq, hs, out_dtype=BF16, **more)
        return (base,) + rmd.sample_block_tokens_processed(base, first, w1, w2, 0.0, **kw, **more)

    def two(h, **more):
        base = rmd.lm_head_logits_int8(h, hq, hs, out_dtype=torch.float32, **more)
        return (base,) + rmd.sample_block_tokens_processed(base, first, w1, w2, 0.6, seed=4, **plain, **more)

    graphs = []
    for f in (one, two):
        f(hidden, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = f(hidden, workspace=ws)
        graphs.append((f, graph, out))
    for k in range(6):
        hidden.copy_(torch.randn(hidden.shape, device="cuda", generator=g))
        kw["history"].copy_(torch.randint(0, V, (B, L), device="cuda", generator=g))
        f, graph, out = graphs[(k + k // 3) % 2]
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, f(hidden.clone())):
            assert torch.equal(got, want)
        f(hidden, workspace=ws)
    assert rmd.read_device_error(ws) == 0


def test_rules_past_31_bits(native):
    """More than 2^31 logits: the last rows are right."""
    B, M, V = 520, 4, 1040001
    assert B * M * V > 2 ** 31
    x = torch.zeros(B, M, V, device="cuda", dtype=BF16)
    x[-1] = torch.randn(M, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(BF16)
    hist = torch.randint(0, V, (B, 100), device="cuda")
    rep = torch.full((B,), 2.0, device="cuda")
    out = rmd.process_block_logits(x, history=hist, repetition_penalty=rep, out=x.clone())
    last = rmd.process_block_logits(x[-1:], history=hist[-1:], repetition_penalty=rep[-1:])
    assert torch.equal(out[-1:], last) and not torch.equal(last, x[-1:])
    back = rmd.process_block_logits_backward(x, x, history=hist, repetition_penalty=rep, out=out.copy_(x))
    assert torch.equal(back[-1:], rmd.process_block_logits_backward(x[-1:], x[-1:], history=hist[-1:], repetition_penalty=rep[-1:]))


@pytest.mark.parametrize("B,M,V,L,r,bias,mask", [
    (64, 5, 8200, 300, 256, "shared", "each"), (17, 3, 16384, 100, 64, "none", "row"), (64, 2, 131064, 40, 16, "none", "none"),
    (33, 16, 520, 60, 32, "shared", "shared"), (5, 4, 40, 9, 8, "none", "each"), (48, 3, 4096, -1, 128, "none", "each")])
def test_greedy_chain_under_rules(native, B, M, V, L, r, bias, mask):
    """Shapes of the persistent greedy chain, and the same draft by steps (as
    fp32 logits would go): its rows and tokens hold by themselves."""
    c = _draft_case(B, M, V, L, r, BF16, BF16, bias=bias, mask=mask, bias_dtype=(F32, BF16)[B % 2])
    ws = rmd.Workspace(B, M, V, r, sample=True, processed=True)
    tok, rows = _draft(c, workspace=ws)
    _check_draft(c, tok, rows)
    again = _draft(c, workspace=ws)                  # the chain leaves the workspace ready
    assert torch.equal(tok, again[0]) and torch.equal(rows, again[1])
    assert rmd.read_device_error(ws) == 0


def test_greedy_chain_with_penalties_far_from_one(native):
    """Repetition penalties whose reciprocal is no number to divide by: with no
    bias in the way the chain's rows are those of the rules alone."""
    rep = torch.tensor([1e-39, 1e-35, 1e35, 3e38, float("inf"), 0.0, 1e-45, 2.0], device="cuda")
    B, M, V, r = len(rep), 1, 1024, 16
    g = torch.Generator(device="cuda").manual_seed(11)
    base = torch.randn(B, M, V, device="cuda", generator=g).to(BF16)
    base[:, :, ::7] = torch.tensor([float("inf"), -float("inf"), 0.0, -0.0, 3e38, 1e-38, float("nan")], device="cuda").to(BF16).repeat(21)
    w = torch.zeros(V, r, dtype=BF16, device="cuda")
    first = torch.zeros(B, dtype=torch.int64, device="cuda")
    kw = dict(history=torch.arange(0, V, 2, device="cuda").repeat(B, 1), repetition_penalty=rep,
              presence_penalty=torch.full((B,), 0.5, device="cuda"))
    _, rows = rmd.sample_block_tokens_processed(base, first, w, w, 0.0, **kw)
    want = rmd.process_block_logits(base, **kw)
    same = (rows == want) | (torch.isnan(rows) & torch.isnan(want))
    assert same.all(), (~same).nonzero()[:5]


def test_greedy_chain_counts_past_a_byte(native):
    """Counts around 254, where the chain's byte ends, and tokens drawn at that edge."""
    B, M, V = 4, 6, 512
    c = _draft_case(B, M, V, 1200, 8, BF16, BF16, mask="none", bias="none")
    c.w1.zero_()
    c.logits.zero_()
    c.logits[:, :, 77] = 200.0                       # drawn whatever its penalties
    c.rep[:] = 1.0
    c.freq[:] = [0.25, 0.125, 0.0625, 0.5]
    c.pres[:] = 0.5
    c.history[:] = 5
    for b, n in enumerate((251, 253, 254, 255)):
        c.history[b, :n] = 77
        c.history[b, n:2 * n + 1] = 78
    c.lengths[:], c.prompt[:] = 1200, [0, 1, 0, 0]
    ws = rmd.Workspace(B, M, V, 8, sample=True, processed=True)
    tok, rows = _draft(c, workspace=ws)
    assert (tok == 77).all()
    _check_draft(c, tok, rows)
    again = _draft(c, workspace=ws)
    assert torch.equal(rows, again[1])


def test_greedy_chain_failure_is_reported(native):
    """A chain whose workgroups do not meet (forced through the workspace's
    hook) gives -1 tokens until the record is read; then it runs again."""
    from rank_markov_draft_amd import _lib
    c = _draft_case(4, 5, 4096, 20, 64, BF16, BF16, mask="none", bias="none")
    ws = rmd.Workspace(4, 5, 4096, 64, sample=True, processed=True)
    want = _draft(c, workspace=ws)
    ws.set_chain_test_hook(True)
    with pytest.raises(_lib.DsparkError, match="DEVICE"):
        _draft(c, workspace=ws, check=True)
    assert (_draft(c, workspace=ws)[0] == -1).all()
    ws.set_chain_test_hook(False)
    assert (_draft(c, workspace=ws)[0] == -1).all()
    with pytest.raises(_lib.DsparkError, match="DEVICE"):
        rmd.read_device_error(ws)
    assert torch.equal(_draft(c, workspace=ws, check=True)[0], want[0])
    again = _draft(c, workspace=ws)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("B", (3, 20))
def test_draft_by_steps_after_a_failed_chain(native, B):
    """A failed chain leaves its own area of the workspace as it stood; drafts
    that run step by step do not read it."""
    from rank_markov_draft_amd import _lib
    c = _draft_case(B, 5, 4096, 20, 64, BF16, BF16, mask="each", bias="row")
    ws = rmd.Workspace(B, 5, 4096, 64, sample=True, processed=True)
    greedy, drawn = _draft(c, workspace=ws), _draft(c, T=0.8, seed=3, workspace=ws)
    plain = (c.logits.cuda(), torch.from_numpy(c.first).cuda(), c.w1.cuda(), c.w2.cuda())
    ws.set_chain_test_hook(True)
    assert (rmd.sample_block_tokens(*plain, 0.0, workspace=ws)[0] == -1).all()
    ws.set_chain_test_hook(False)
    for _ in range(2):
        for want, got in ((greedy, _draft(c, workspace=ws)), (drawn, _draft(c, T=0.8, seed=3, workspace=ws))):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(_lib.DsparkError, match="DEVICE"):
        rmd.read_device_error(ws)
    again = _draft(c, workspace=ws)
    assert torch.equal(again[0], greedy[0]) and torch.equal(again[1], greedy[1])


def test_draft_of_more_rows_than_the_keys_hold(native):
    """70000 requests: their best keys do not fit beside the counters, so a
    second launch reduces them; the same rows in smaller calls are the same."""
    B, V, r = 70000, 40, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    base = torch.randn(B, 2, V, device="cuda", generator=g)
    w1, w2 = (torch.randn(V, r, device="cuda", generator=g) * 0.1 for _ in range(2))
    first = torch.randint(0, V, (B,), device="cuda", generator=g)
    hist = torch.randint(0, V, (B, 5), device="cuda", generator=g)
    rep = 1.0 + torch.rand(B, device="cuda", generator=g)
    tok, rows = rmd.sample_block_tokens_processed(base, first, w1, w2, 0.6, history=hist, repetition_penalty=rep, seed=8)
    for a, b in ((0, 300), (35000, 36000), (69000, 70000)):
        t, x = rmd.sample_block_tokens_processed(base[a:b], first[a:b], w1, w2, 0.6, history=hist[a:b],
                                                 repetition_penalty=rep[a:b], seed=8, batch_offset=a)
        assert torch.equal(t, tok[a:b]) and torch.equal(x, rows[a:b])
