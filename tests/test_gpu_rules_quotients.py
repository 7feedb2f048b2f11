"""The repetition penalty's quotient in the greedy chain is the division's own:
without a bias the chain's rows are those of process_block_logits, which
divides."""
import pytest
import torch

import rank_markov_draft_amd as rmd

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _same(a, b):
    return (a == b) | (torch.isnan(a) & torch.isnan(b))


def _chain_and_rules(base, **kw):
    """(tokens, rows) of a draft that runs in the greedy chain and has no bias, and the rules on its logits."""
    B, M, V = base.shape
    w = torch.zeros(V, 16, dtype=BF16, device="cuda")
    first = torch.zeros(B, dtype=torch.int64, device="cuda")
    ws = rmd.Workspace(B, M, V, 16, sample=True, processed=True)
    tok, rows = rmd.sample_block_tokens_processed(base, first, w, w, 0.0, workspace=ws, check=True, **kw)
    return tok, rows, rmd.process_block_logits(base, **kw)


PENALTIES = [0.5, 0.99, 0.999999, 1.0 / 3.0, 0.7, 0.1, 1e-3, 1e-20, 1e-29, 1.0, 1.0000001, 1.0001, 1.05, 1.1, 1.15, 1.2, 1.25,
             1.3, 4.0 / 3.0, 1.4, 1.5, 1.7, 1.9999999, 2.0, 2.5, 3.0, 5.0, 7.77, 10.0, 100.0, 1023.0, 1e6, 1e7, 1e12, 1e25,
             1e30, float.fromhex("0x1.a15686p+0"), float.fromhex("0x1.f250c6p+0"), float.fromhex("0x1.f250c6p-3")]


@pytest.mark.parametrize("first", [0, 20])
def test_every_bf16_value(native, first):
    """All 65536 bit patterns as one row, under many penalties."""
    V = 65536
    reps = PENALTIES[first:first + 20]
    base = torch.arange(V, dtype=torch.int32).to(torch.int16).view(BF16).cuda().expand(len(reps), 1, V).contiguous()
    every = torch.arange(V, device="cuda").repeat(len(reps), 1)
    for counted in (dict(), dict(frequency_penalty=torch.full((len(reps),), 0.25, device="cuda"))):
        _, rows, want = _chain_and_rules(base, history=every, repetition_penalty=torch.tensor(reps, device="cuda"), **counted)
        same = _same(rows, want).reshape(len(reps), V)
        bad = [(reps[int(b)], base[0, 0, int(v)].item(), rows[int(b), 0, int(v)].item(), want[int(b), 0, int(v)].item())
               for b, v in (~same).nonzero()[:5]]
        assert same.all(), (int((~same).sum()), bad)


def test_drawn_penalties(native):
    """64 penalties a call between 1 and 2 and between one half and 1, on every bf16 value of the logits' usual range."""
    values = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    values = values[(values.float().abs() < 256.0) & (values.float().abs() > 2.0 ** -20)]
    V = values.numel() // 8 * 8
    base = values[:V].cuda().expand(64, 1, V).contiguous()
    every = torch.arange(V, device="cuda").repeat(64, 1)
    for seed in range(6):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rep = 1.0 + torch.rand(64, device="cuda", generator=g) * (1.0 if seed % 2 else -0.5)
        _, rows, want = _chain_and_rules(base, history=every, repetition_penalty=rep)
        assert torch.equal(rows, want), int((rows != want).sum())


def test_quotients_past_the_type_are_infinite(native):
    """3e38 / 0.5 and the type's largest value over 0.99 are infinite, not
    NaN, and do not take the draw from an infinity before them."""
    big = torch.finfo(BF16).max
    V, reps = 512, [0.5, 0.99, 0.5, 0.99]
    base = torch.zeros(4, 1, V, dtype=BF16, device="cuda")
    base[0, 0, 40], base[1, 0, 40] = 3e38, big
    base[2:, 0, 40] = float("inf")
    base[2, 0, 300], base[3, 0, 300] = 3e38, big
    every = torch.arange(V, device="cuda").repeat(4, 1)
    kw = dict(history=every, repetition_penalty=torch.tensor(reps, device="cuda"))
    tok, rows, want = _chain_and_rules(base, **kw)
    assert tok[:, 0].tolist() == [40] * 4
    assert not torch.isnan(rows).any() and (rows[torch.arange(4), 0, [40, 40, 300, 300]] == float("inf")).all()
    assert torch.equal(rows, want)
