"""The 4-bit head, sampling under limits and distillation with one workspace
between them, in captured graphs that share it, and on two streams at once."""
import pytest
import torch

import rank_markov_draft_amd as rmd

pytestmark = pytest.mark.gpu

B, M, V, D, K = 6, 3, 9001, 320, 12


def _gen(seed):
    return dict(device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


class Case:
    """Inputs of all three operators, and their calls."""

    def __init__(self, seed):
        self.hc, self.hs = rmd.quantize_blocks_fp4(0.1 * torch.randn(V, D, **_gen(90)))
        self.x = torch.empty(B, M, D, device="cuda")
        self.logits = torch.empty(B, M, V, device="cuda")
        self.u = torch.empty(B, M, device="cuda")
        self.ids = torch.empty(B, M, K, dtype=torch.int64, device="cuda")
        self.t = torch.empty(B, M, K, device="cuda")
        self.fill(seed)

    def fill(self, seed):
        self.x.copy_(torch.randn(B, M, D, **_gen(seed)))
        self.logits.copy_(2 * torch.randn(B, M, V, **_gen(seed + 1)))
        self.u.copy_(torch.rand(B, M, **_gen(seed + 2)))
        self.ids.copy_(torch.rand(B, M, V, **_gen(seed + 3)).topk(K).indices)
        self.t.copy_(torch.randn(B, M, K, **_gen(seed + 4)))

    def head(self, ws=None):
        return [rmd.lm_head_logits_fp4(self.x, self.hc, self.hs, workspace=ws)]

    def sample(self, ws=None):
        return list(rmd.sample_block_filtered(self.logits, self.u, 0.8, top_k=2500, top_p=0.95, workspace=ws))

    def distill(self, ws=None):
        loss, stats = rmd.distill_block_loss(self.logits, self.ids, self.t, workspace=ws)
        return [loss, rmd.distill_block_loss_backward(torch.ones_like(loss), self.logits, self.ids, self.t, stats)]


def _same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_one_workspace_in_turn(native):
    c = Case(1)
    want = [c.head(), c.sample(), c.distill()]
    ws = rmd.Workspace(B, M, V, 1, sample=False, fp4_hidden=D, distill=True, filtered=True)
    for _ in range(3):
        for call, w in zip((c.head, c.sample, c.distill), want):
            assert _same(call(ws), w)


@pytest.mark.parametrize("T", [0.0, 0.8])
@pytest.mark.parametrize("dtype,v", [(torch.bfloat16, 9008), (torch.float32, 9001)])
def test_drafts_between_them(native, dtype, v, T):
    """Drafts, with and without rules, on the workspace that the others have written."""
    c = Case(50)
    want = [c.head(), c.sample(), c.distill()]
    w1, w2 = (0.1 * torch.randn(v, 64, **_gen(s)).to(dtype) for s in (51, 52))
    base = torch.randn(B, M, v, **_gen(53)).to(dtype)
    first = torch.randint(0, v, (B,), **_gen(54))
    history = torch.randint(0, v, (B, 40), **_gen(55))
    rep = torch.full((B,), 1.3, device="cuda")

    def drafts(**kw):
        return [*rmd.sample_block_tokens(base, first, w1, w2, temperature=T, seed=3, **kw),
                *rmd.sample_block_tokens_processed(base, first, w1, w2, temperature=T, seed=3, history=history,
                                                   repetition_penalty=rep, **kw)]

    plain = drafts()
    ws = rmd.Workspace(B, M, 9008, 64, sample=True, processed=True, fp4_hidden=D, distill=True, filtered=True)
    for turn in range(3):
        for call, w in zip((c.head, c.sample, c.distill), want):
            assert _same(call(ws), w), turn
            assert _same(drafts(workspace=ws), plain), turn
    assert rmd.read_device_error(ws) == 0


@pytest.mark.parametrize("name", ["head", "sample", "distill"])
def test_graphs_share_a_workspace(native, name):
    ws = rmd.Workspace(B, M, V, 1, sample=False, fp4_hidden=D, distill=True, filtered=True)
    cases = [Case(10), Case(20)]
    graphs, results = [], []
    for c in cases:
        getattr(c, name)(ws)
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(getattr(c, name)(ws))
        graphs.append(graph)
    for turn in range(4):
        for i, c in enumerate(cases):
            c.fill(100 * turn + 10 * i)
        for i in (0, 1) if turn % 2 else (1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        for c, r in zip(cases, results):
            assert _same(r, getattr(c, name)()), turn


def test_two_streams_at_once(native):
    cases = [Case(30), Case(40)]
    want = [[c.head(), c.sample(), c.distill()] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for turn in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append([cases[i].head(), cases[i].sample(), cases[i].distill()])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for turn in g:
            for a, b in zip(turn, w):
                assert _same(a, b)
