"""The largest vocabularies that the calls take: 2^30 columns under the rules,
2^31 - 1 in the 8-bit head."""
import pytest
import torch

import rank_markov_draft_amd as rmd

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def room(native):
    yield
    torch.cuda.empty_cache()


def _mask(V):
    """Every token but 4, V - 3 and one in the middle."""
    words = torch.full((1, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    for v in (4, V - 3, V // 2):
        bit = 1 << v % 32
        words[0, v // 32] = (words[0, v // 32].item() & 0xFFFFFFFF & ~bit) - (0 if bit == 1 << 31 else 1 << 32)
    return words


@pytest.mark.parametrize("V", [2 ** 30, 2 ** 30 - 5])
def test_rules(native, V):
    x = torch.ones(1, 1, V, dtype=BF16, device="cuda")
    ids = torch.tensor([[1, V - 2, V - 1, V - 1, V // 2 + 1, V, -1]], device="cuda")
    kw = dict(history=ids, repetition_penalty=torch.tensor([2.0], device="cuda"), token_mask=_mask(V))
    out = rmd.process_block_logits(x, prompt_lengths=torch.tensor([2], device="cuda"),
                                   frequency_penalty=torch.tensor([0.25], device="cuda"), **kw)
    back = rmd.process_block_logits_backward(x, x, **kw)
    want = {1: 0.5, V - 2: 0.5, V - 1: 0.0, V // 2 + 1: 0.25, 4: -float("inf"), V - 3: -float("inf"), V // 2: -float("inf")}
    for v, value in want.items():
        assert out[0, 0, v].item() == value
        assert back[0, 0, v].item() == (0.0 if value == -float("inf") else 0.5)
        out[0, 0, v], back[0, 0, v] = 1.0, 1.0
    assert (out == 1).all() and (back == 1).all()


@pytest.mark.parametrize("T", [0.0, 0.5])
@pytest.mark.parametrize("r", [1, 8])
def test_drafts(native, r, T):
    """Few rows (rank 8) and row tiles (rank 1); the drawn tokens lie at the end."""
    V, M = 2 ** 30 - 5, 3
    x = torch.zeros(1, M, V, dtype=BF16, device="cuda")
    x[:, :, V - 1], x[:, :, V - 3], x[:, :, V // 2 + 1] = 300.0, 400.0, 200.0
    w1 = torch.zeros(V, r, dtype=BF16, device="cuda")
    w2 = torch.zeros(V, r, dtype=BF16, device="cuda")
    w1[V - 1], w2[V // 2 + 1], w2[V - 2] = 1.0, 150.0 / r, 1.0 / r   # after V - 1 the middle holds 350
    ws = rmd.Workspace(1, M, V, r, sample=True, processed=True)
    tok, out = rmd.sample_block_tokens_processed(
        x, torch.tensor([0], device="cuda"), w1, w2, T, history=torch.tensor([[7]], device="cuda"),
        presence_penalty=torch.tensor([250.0], device="cuda"), token_mask=_mask(V), workspace=ws)
    assert tok.tolist() == [[V - 1, V // 2 + 1, V - 1]]
    assert out[0, 1, V - 2].item() == 1.0 and out[0, 1, V - 1].item() == 50.0 and out[0, 1, V // 2 + 1].item() == 350.0
    assert out[0, 2, V // 2 + 1].item() == -50.0 and out[0, 0, V - 3].item() == -float("inf")


@pytest.mark.parametrize("d", [1, 4])
def test_int8_head(native, d):
    V = 2 ** 31 - 1
    hq = torch.ones(V, d, dtype=torch.int8, device="cuda")
    hs = torch.ones(V, device="cuda")
    hq[V - 1], hq[2 ** 30 + 7], hs[V - 2] = -3, 5, 2.0
    out = rmd.lm_head_logits_int8(torch.full((1, d), 127.0, device="cuda"), hq, hs, out_dtype=BF16)
    one = 127.0 * d
    want = {V - 1: -3 * one, 2 ** 30 + 7: 5 * one, V - 2: 2 * one}
    for v, value in want.items():
        assert out[0, v].item() == torch.tensor(value).to(BF16).item()
        out[0, v] = one
    assert (out == torch.tensor(one).to(BF16).item()).all()
