"""More rows and requests than one launch takes workgroups: a launch ends at
2^32 - 1 threads, 2^24 - 1 workgroups of 256."""
import pytest
import torch

import rank_markov_draft_amd as rmd

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _gen(seed):
    return dict(device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


@pytest.mark.parametrize("rows,d,dtype", [(2 ** 24 + 5, 3, F32), (2 ** 24 + 5, 5, BF16), (2 ** 26 + 3, 8, BF16)])
def test_quantize_more_rows_than_a_launch(native, rows, d, dtype):
    """Rows of odd length go one to a workgroup, short whole ones four."""
    x = torch.randn(rows, d, dtype=dtype, **_gen(d))
    q, s = rmd.quantize_rows(x)
    edge = 2 ** 24 - 1 if d % 8 else 4 * (2 ** 24 - 1)
    for a, b in ((0, 9), (edge - 9, edge + 9), (rows - 9, rows)):
        wq, ws = rmd.quantize_rows(x[a:b].clone())
        assert torch.equal(q[a:b], wq) and torch.equal(s[a:b], ws) and ws.all()
    n = 1 << 22
    for a in range(0, rows, n):                      # every row was written
        assert (q[a:a + n].abs().amax(-1) == 127).all()


def test_rules_of_more_requests_than_a_launch(native):
    B, V, L = 2 ** 24 + 5, 5, 3
    x = torch.randn(B, 1, V, dtype=BF16, **_gen(1))
    history = torch.randint(0, V, (B, L), **_gen(2))
    rep, pres = 1.0 + torch.rand(B, **_gen(3)), torch.rand(B, **_gen(4))
    mask = torch.randint(0, 32, (B, 1), **_gen(5)).int()
    bias = torch.randn(B, V, **_gen(6))
    g = torch.randn(B, 1, V, dtype=BF16, **_gen(7))
    fwd = rmd.process_block_logits(x, history=history, repetition_penalty=rep, presence_penalty=pres, logit_bias=bias, token_mask=mask)
    back = rmd.process_block_logits_backward(g, x, history=history, repetition_penalty=rep, token_mask=mask)
    for a, b in ((0, 9), (2 ** 24 - 9, 2 ** 24 + 4), (B - 9, B)):
        assert torch.equal(fwd[a:b], rmd.process_block_logits(x[a:b], history=history[a:b], repetition_penalty=rep[a:b],
                                                              presence_penalty=pres[a:b], logit_bias=bias[a:b], token_mask=mask[a:b]))
        assert torch.equal(back[a:b], rmd.process_block_logits_backward(g[a:b], x[a:b], history=history[a:b],
                                                                        repetition_penalty=rep[a:b], token_mask=mask[a:b]))


def test_drafts_of_more_requests_than_a_launch(native):
    B, V, r = 2 ** 24 + 5, 8, 4
    x = torch.randn(B, 2, V, dtype=BF16, **_gen(1))
    w1, w2 = (torch.randn(V, r, **_gen(8 + i)).to(BF16) for i in range(2))
    first = torch.randint(0, V, (B,), **_gen(2))
    history, rep = torch.randint(0, V, (B, 2), **_gen(3)), 1.0 + torch.rand(B, **_gen(4))
    tok, rows = rmd.sample_block_tokens_processed(x, first, w1, w2, 0.7, history=history, repetition_penalty=rep, seed=2)
    for a, b in ((0, 70), (2 ** 24 - 70, 2 ** 24 + 4), (B - 70, B)):
        t, o = rmd.sample_block_tokens_processed(x[a:b], first[a:b], w1, w2, 0.7, history=history[a:b],
                                                 repetition_penalty=rep[a:b], seed=2, batch_offset=a)
        assert torch.equal(t, tok[a:b]) and torch.equal(o, rows[a:b])
