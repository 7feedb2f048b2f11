"""A batch split across calls reproduces the whole call under the rules, bit
for bit: the form that a size picks does not change a row."""
import pytest
import torch

import rank_markov_draft_amd as rmd

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _inputs(B, M, V, r, ldt, wdt, L=40):
    g = torch.Generator(device="cuda").manual_seed(B + V + r)
    kw = dict(device="cuda", generator=g)
    x = (torch.randn(B, M, V, **kw) * 2).to(ldt)
    w1, w2 = ((torch.randn(V, r, **kw) * 0.2).to(wdt) for _ in range(2))
    rows = dict(first_prev_token_ids=torch.randint(0, V, (B,), **kw), history=torch.randint(0, V, (B, L), **kw),
                lengths=torch.randint(0, L + 1, (B,), **kw), prompt_lengths=torch.randint(0, L, (B,), **kw),
                repetition_penalty=0.8 + torch.rand(B, **kw), frequency_penalty=torch.rand(B, **kw),
                presence_penalty=torch.rand(B, **kw),
                token_mask=torch.randint(-2 ** 31, 2 ** 31, (B, M, (V + 31) // 32), dtype=torch.int64, **kw).int())
    shared = dict(logit_bias=torch.randn(V, **kw), w1=w1, w2=w2, seed=11)
    return x, rows, shared


def _draft(x, rows, shared, T, a, b, k=None):
    at = slice(None) if k is None else slice(k, k + 1)
    part = {n: t[a:b, at] if n == "token_mask" else t[a:b] for n, t in rows.items()}
    return rmd.sample_block_tokens_processed(x[a:b, at], temperature=T, batch_offset=a, position_offset=k or 0, **part, **shared)


@pytest.mark.parametrize("T", [0.0, 0.7])
@pytest.mark.parametrize("B,V,r,ldt,wdt", [
    (16, 40000, 64, F32, F32), (16, 40000, 64, BF16, F32), (24, 40000, 32, F32, BF16), (70, 1000, 64, F32, F32),
    (70, 1000, 16, F32, BF16), (70, 1024, 64, BF16, BF16), (70, 1001, 50, BF16, BF16), (65, 515, 100, F32, F32),
    (300, 264, 33, F32, F32), (300, 264, 40, BF16, BF16), (130, 333, 7, BF16, BF16), (130, 333, 300, F32, F32),
    (80, 2048, 256, BF16, BF16), (96, 640, 512, BF16, BF16), (100, 999, 258, F32, BF16), (100, 300, 1000, F32, F32)])
def test_pieces_of_a_batch(native, B, V, r, ldt, wdt, T):
    """Pieces of 64, 16, 4 rows and one: row tiles, four rows a workgroup, and
    in bf16 the greedy chain."""
    M = 3
    x, rows, shared = _inputs(B, M, V, r, ldt, wdt)
    tok, out = _draft(x, rows, shared, T, 0, B)
    for size in (64, 16, 4, 1):
        for a in range(0, B, size) if size > 4 else (0, 4 * ((B - 1) // 4), B - 1):
            b = min(B, a + size)
            t, o = _draft(x, rows, shared, T, a, b)
            assert torch.equal(o, out[a:b]), f"rows {a} .. {b}: {int((o != out[a:b]).sum())} differ"
            assert torch.equal(t, tok[a:b])


@pytest.mark.parametrize("T", [0.0, 0.7])
@pytest.mark.parametrize("B,V,r,ldt,wdt", [(5, 1001, 100, F32, F32), (20, 40000, 64, F32, BF16), (70, 1000, 40, BF16, BF16),
                                           (64, 4096, 64, BF16, BF16)])
def test_a_shared_bias_and_one_for_each_request(native, B, V, r, ldt, wdt, T):
    """The greedy chain takes shared biases only: the same biases given for
    each request run step by step, with the same rows."""
    x, rows, shared = _inputs(B, 3, V, r, ldt, wdt)
    want = _draft(x, rows, shared, T, 0, B)
    got = _draft(x, rows, dict(shared, logit_bias=shared["logit_bias"].expand(B, V).contiguous()), T, 0, B)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("r", [1, 3, 4, 7, 8, 15, 16, 17, 24, 31, 32, 33, 40, 63, 64, 65, 72, 95, 96, 127, 128, 129, 160, 255, 256, 264, 511, 520])
def test_every_rank(native, r):
    """Ranks on both sides of a vector, a product's depth, a line and a chunk."""
    V = 200
    for ldt, wdt in ((F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)):
        x, rows, shared = _inputs(66, 2, V, r, ldt, wdt, L=5)
        tok, out = _draft(x, rows, shared, 0.6, 0, 66)
        for a, b in ((0, 4), (4, 66), (65, 66)):
            t, o = _draft(x, rows, shared, 0.6, a, b)
            assert torch.equal(t, tok[a:b]) and torch.equal(o, out[a:b]), (ldt, wdt, a)
