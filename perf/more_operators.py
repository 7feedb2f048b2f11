"""What is measured of the 4-bit vocabulary head, of sampling under a
request's limits (temperature, top-k, top-p, min-p) and of distillation from a
teacher's top logits.

Each case names an operator (``op``) and its sizes.  With ``own`` false,
``run`` computes the operators with elementary torch operations; with ``own``
true it makes the calls of the framework.
"""
import math

import torch

own = False

F32, BF16 = "float32", "bfloat16"


def listed():
    return [
        # blocks of 32 numbers as 4-bit codes with a shared power of two, and
        # back: one decode batch of hidden states, and the head's own weight
        # when a server loads it
        dict(name="fp4 quantize hidden 64", op="quantize", rows=64, d=5120, dtype=BF16),
        dict(name="fp4 quantize head", op="quantize", rows=129280, d=5120, dtype=BF16),
        # the head: a single token, a verified block of 64 requests, a ragged
        # batch on a small odd vocabulary, a training-sized batch of blocks
        dict(name="fp4 head 1 token", op="head", rows=1, d=5120, V=129280, dtype=BF16, out=F32),
        dict(name="fp4 head 64x5", op="head", rows=320, d=5120, V=129280, dtype=BF16, out=F32),
        dict(name="fp4 head odd", op="head", rows=37, d=2056, V=32003, dtype=F32, out=BF16),
        dict(name="fp4 head 512x5", op="head", rows=2560, d=5120, V=129280, dtype=BF16, out=BF16),
        # sampling: one request with every limit on; a served batch in which
        # each request brings its own limits, half of them inside a grammar;
        # a large batch of nucleus sampling on fp32 logits
        dict(name="sample 1 token", op="sample", B=1, M=1, V=129280, dtype=BF16, limits="all", mask=False),
        dict(name="sample 64x5", op="sample", B=64, M=5, V=129280, dtype=BF16, limits="mixed", mask=True),
        dict(name="sample 256x8", op="sample", B=256, M=8, V=151936, dtype=F32, limits="top_p", mask=False),
        # distillation, the loss and the gradient of the drafter's logits: a
        # few blocks on an odd vocabulary, the 320-row batch, and 512 blocks
        # of 8 positions with a long list from the teacher
        dict(name="distill 2x4", op="distill", B=2, M=4, V=50257, K=20, dtype=F32, tau=2.0),
        dict(name="distill 64x5", op="distill", B=64, M=5, V=129280, K=64, dtype=BF16, tau=1.0),
        dict(name="distill 512x8", op="distill", B=512, M=8, V=129280, K=128, dtype=BF16, tau=1.0),
    ]


LIMITS = ["greedy", "none", "top_k", "top_p", "min_p", "all"]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "head", "head", "sample", "sample", "distill", "distill"])
    dt = rng.choice([F32, BF16])
    if op == "quantize":
        return dict(op=op, rows=_spread(rng, 1, 60000), d=_spread(rng, 64, 5120), dtype=dt)
    if op == "head":
        d = _spread(rng, 64, 5120)
        if rng.random() < 0.6:
            d = (d + 63) // 64 * 64
        return dict(op=op, rows=_spread(rng, 1, 2000), d=d, V=_spread(rng, 1000, 129280), dtype=dt,
                    out=rng.choice([F32, BF16]))
    V = _spread(rng, 1000, 151936)
    if rng.random() < 0.5:
        V = (V + 7) // 8 * 8
    c = dict(op=op, B=_spread(rng, 1, 200), M=rng.randint(1, 8), V=V, dtype=dt)
    if op == "sample":
        c.update(limits=rng.choice(["mixed", "mixed", "none", "top_k", "top_p", "min_p", "all"]),
                 mask=rng.random() < 0.4)
    else:
        c.update(K=_spread(rng, 1, 256), tau=rng.choice([1.0, 0.5, 2.0]))
    return c


def _dtype(name):
    return torch.float32 if name == F32 else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    s = dict(case)
    op = case["op"]
    if op in ("quantize", "head"):
        # activations and weights: normal, a few channels larger than the rest
        rows, d = case["rows"], case["d"]
        channel = torch.where(uniform(d) < 0.02, 6.0, 1.0)
        s["x"] = (normal(rows, d) * channel).to(_dtype(case["dtype"]))
        if op == "head":
            V, B = case["V"], (d + 127) // 128 * 4
            s["codes"] = torch.empty(V, 16 * B, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(V, B, dtype=torch.uint8, device="cuda")
            for v in range(0, V, 16384):
                codes, scales = _fp4(0.02 * normal(min(V, v + 16384) - v, d))
                s["codes"][v:v + 16384] = codes[:, ::2] | (codes[:, 1::2] << 4)
                s["scales"][v:v + 16384] = scales
        return s
    B, M, V = case["B"], case["M"], case["V"]
    x = normal(B, M, V).mul_(2.0)
    if op == "sample":
        # a position with two dozen plausible tokens
        x.scatter_add_(2, (uniform(B, M, 24) * V).long(), 12.0 * uniform(B, M, 24))
        if case["mask"]:  # every other request inside a grammar; the last row of a batch at its end
            x[::2].masked_fill_(uniform((B + 1) // 2, M, V) < 0.9, -math.inf)
            if B > 7:
                x[-1, -1] = -math.inf
        s["logits"] = x.to(_dtype(case["dtype"]))
        s["uniforms"] = uniform(B, M)
        kind = [LIMITS[b % len(LIMITS)] if case["limits"] == "mixed" else case["limits"] for b in range(B)]

        def only(values, off, *kinds):
            on = torch.tensor([k in kinds for k in kind], device="cuda")
            return torch.where(on, values, off)

        s["temperature"] = only((0.5 + 0.7 * uniform(B)), 0.0, *LIMITS[1:])
        s["top_k"] = only((20 + 80 * uniform(B)).long(), 0, "top_k", "all")
        s["top_p"] = only(0.8 + 0.19 * uniform(B), 1.0, "top_p", "all")
        s["min_p"] = only(0.02 + 0.1 * uniform(B), 0.0, "min_p", "all")
        return s
    # distillation: the teacher agrees with the drafter up to noise; some of
    # its lists are shorter than the others, one row has none (a padded
    # position); the loss is weighted by position
    K = case["K"]
    s["logits"] = x.to(_dtype(case["dtype"]))
    chunks = [torch.topk(c + normal(*c.shape), K, dim=-1) for c in x.reshape(B * M, V).split(512)]
    s["teacher_logits"] = torch.cat([c.values for c in chunks]).to(s["logits"].dtype).reshape(B, M, K)
    s["teacher_ids"] = torch.cat([c.indices for c in chunks]).reshape(B, M, K)
    short = (torch.arange(K, device="cuda") >= 3 * K // 4) & (uniform(B, M, 1) < 0.25)
    s["teacher_ids"][short] = -1
    if B > 1:
        s["teacher_ids"][-1, -1] = -1
    s["grad_loss"] = torch.exp(-0.25 * torch.arange(M, device="cuda")).expand(B, M) / (B * M)
    s["grad_loss"] = s["grad_loss"] * (uniform(B, M) + 0.5)
    return s


# ------------------------------------------------------------ plain forms
_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exponent(x):
    """floor(log2 x) of positive numbers, exactly (x a 32-bit float)."""
    return torch.frexp(x).exponent - 1


def _fp4(x):
    """Codes 0..15 [rows, 32 blocks] (sign in bit 3) and biased exponents [rows, blocks] of x [rows, d]."""
    rows, d = x.shape
    blocks = (d + 127) // 128 * 4
    p = torch.zeros(rows, 32 * blocks, device=x.device)
    p[:, :d] = x
    p = p.view(rows, blocks, 32)
    top = p.abs().amax(-1)
    e = torch.where(top > 0, _exponent(top) - 2, -127).clamp(-127, 127)
    # x / 2^e in two exact steps: 2^-e alone may leave the range
    half = e // 2
    y = torch.ldexp(torch.ldexp(p.abs(), -half[..., None]), -(e - half)[..., None])
    # the step below 2 is 1/2, below 4 it is 1, above it is 2; torch.round takes ties to even
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp_(max=6.0)
    code = torch.bucketize(y, torch.tensor(_VALUES, device=x.device))
    code = code + 8 * (p < 0)
    return code.to(torch.uint8).view(rows, 32 * blocks), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """The numbers of codes [rows, 32 blocks] with biased exponents [rows, blocks], fp32."""
    table = torch.tensor(_VALUES + [-v for v in _VALUES], device=codes.device)
    e = scales.int() - 127
    half = e // 2
    y = table[codes.int()].view(codes.shape[0], -1, 32)
    return torch.ldexp(torch.ldexp(y, half[..., None]), (e - half)[..., None]).view(codes.shape)


def _quantize(s):
    d = s["x"].shape[1]
    out = torch.empty_like(s["x"])
    for r in range(0, out.shape[0], 16384):  # a 16th of the head at a time
        out[r:r + 16384] = _values(*_fp4(s["x"][r:r + 16384].float()))[:, :d].to(out.dtype)
    return out


def _head(s):
    x = _values(*_fp4(s["x"].float()))
    V = s["codes"].shape[0]
    y = torch.empty(x.shape[0], V, device="cuda", dtype=_dtype(s["out"]))
    for v in range(0, V, 32768):
        c = s["codes"][v:v + 32768]
        w = _values(torch.stack([c & 15, c >> 4], -1).view(c.shape[0], -1), s["scales"][v:v + 32768])
        y[:, v:v + 32768] = (x @ w.t()).to(y.dtype)
    return y


def _sample_rows(x, u, T, k, p, m):
    """Tokens and probabilities of rows x [n, V]: weights and sums in 64 bits, whose borders decide the tokens."""
    V = x.shape[1]
    value, order = torch.sort(x, dim=-1, descending=True, stable=True)
    greedy = T < 1e-5
    T = torch.where(greedy, 1.0, T.double())[:, None]
    w = torch.exp((value.double() - value[:, :1].double()) / T)
    w = torch.where(value == -math.inf, 0.0, w)
    rank = torch.arange(V, device=x.device)
    k = torch.where(greedy, 1, torch.where(k <= 0, V, k))[:, None]
    w = torch.where((rank < k) & (w >= m.double()[:, None]), w, 0.0)
    upto = w.cumsum(-1)
    reach = (upto - w < p.double()[:, None] * upto[:, -1:]) | (p[:, None] >= 1) | (rank == 0)
    w = torch.zeros_like(w).scatter_(1, order, torch.where(reach, w, 0.0))
    upto = w.cumsum(-1)
    at = torch.searchsorted(upto, u.double()[:, None] * upto[:, -1:], right=True).clamp_(max=V - 1)
    prob = torch.gather(w, 1, at) / upto[:, -1:]
    some = value[:, 0] > -math.inf
    return torch.where(some, at[:, 0], -1), torch.where(some, prob[:, 0], 0.0).float()


def _sample(s):
    B, M, V = s["logits"].shape
    x, u = s["logits"].reshape(B * M, V), s["uniforms"].reshape(-1)
    limits = [s[n].repeat_interleave(M) for n in ("temperature", "top_k", "top_p", "min_p")]
    step = max(1, (1 << 27) // V)
    parts = [_sample_rows(x[r:r + step].float(), u[r:r + step], *(t[r:r + step] for t in limits))
             for r in range(0, B * M, step)]
    return {"tokens": torch.cat([t for t, _ in parts]).view(B, M), "probs": torch.cat([q for _, q in parts]).view(B, M)}


def _distill(s):
    tau, V = s["tau"], s["logits"].shape[-1]
    ids, t = s["teacher_ids"], s["teacher_logits"].float() / tau
    ok = (ids >= 0) & (ids < V)
    some = ok.any(-1, keepdim=True)
    t = torch.where(ok, t, -math.inf)
    top = torch.where(some, t.amax(-1, keepdim=True), 0.0)
    q = torch.exp(t - top)
    total = torch.where(some, q.sum(-1, keepdim=True), 1.0)
    q = q / total
    logq = torch.where(ok, t - top - torch.log(total), 0.0)
    x = s["logits"].float() / tau
    x = x - x.amax(-1, keepdim=True)
    e = torch.exp(x)
    sums = e.sum(-1, keepdim=True)
    safe = torch.where(ok, ids, 0)
    logp = torch.gather(x, -1, safe) - torch.log(sums)
    loss = tau * tau * (q * (logq - logp)).sum(-1)
    grad = e.div_(sums).scatter_add_(-1, safe, -q)
    grad *= torch.where(some, s["grad_loss"][..., None] * tau, 0.0)
    return {"loss": torch.where(some[..., 0], loss, 0.0), "grad": grad.to(s["logits"].dtype)}


# ------------------------------------------------------------ one pass
def _own(s):
    import rank_markov_draft_amd as rmd

    op = s["op"]
    if op == "quantize":
        codes, scales = rmd.quantize_blocks_fp4(s["x"])
        return {"values": rmd.dequantize_blocks_fp4(codes, scales, s["d"], dtype=s["x"].dtype)}
    if op == "head":
        if "workspace" not in s:  # a server keeps it beside its weights
            s["workspace"] = rmd.Workspace(s["rows"], 1, s["V"], 1, sample=False, fp4_hidden=s["d"])
        return {"logits": rmd.lm_head_logits_fp4(s["x"], s["codes"], s["scales"], out_dtype=_dtype(s["out"]),
                                                 workspace=s["workspace"])}
    B, M, V = s["logits"].shape
    if op == "sample":
        if "workspace" not in s:
            s["workspace"] = rmd.Workspace(B, M, V, 1, sample=False, filtered=True)
        tokens, probs = rmd.sample_block_filtered(s["logits"], s["uniforms"], s["temperature"], top_k=s["top_k"],
                                                  top_p=s["top_p"], min_p=s["min_p"], workspace=s["workspace"])
        return {"tokens": tokens, "probs": probs}
    if "workspace" not in s:  # as a trainer does, for all its steps
        s["workspace"] = rmd.Workspace(B, M, V, 1, sample=False, distill=True)
    loss, stats = rmd.distill_block_loss(s["logits"], s["teacher_ids"], s["teacher_logits"], temperature=s["tau"],
                                         workspace=s["workspace"])
    grad = rmd.distill_block_loss_backward(s["grad_loss"], s["logits"], s["teacher_ids"], s["teacher_logits"], stats,
                                           temperature=s["tau"])
    return {"loss": loss, "grad": grad}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "quantize":
        return {"values": _quantize(state)}
    if op == "head":
        return {"logits": _head(state)}
    if op == "sample":
        return _sample(state)
    return _distill(state)


def work(case):
    size = {F32: 4, BF16: 2}
    op, es = case["op"], size[case["dtype"]]
    if op == "quantize":
        return {"bytes": 2 * case["rows"] * case["d"] * es, "flops": 0}
    if op == "head":
        rows, d, V = case["rows"], case["d"], case["V"]
        return {"bytes": V * d * 17 // 32 + rows * d * es + rows * V * size[case["out"]], "flops": 2 * rows * d * V}
    rows, V = case["B"] * case["M"], case["V"]
    if op == "sample":
        return {"bytes": rows * V * es + rows * 16 + case["B"] * 20, "flops": 0}
    return {"bytes": 2 * rows * V * es + rows * (case["K"] * (8 + es) + 8), "flops": 0}


# ------------------------------------------------------------ in 64 bits
def _exact_blocks(x):
    """The nearest of the fifteen numbers at each block's scale, by distance, [rows, d] in 64 bits."""
    rows, d = x.shape
    out = torch.zeros(rows, d, device=x.device, dtype=torch.float64)
    table = torch.tensor(_VALUES, device=x.device, dtype=torch.float64)
    # the value with the even code first wins a tie: the even codes before the odd ones
    table = table[torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=x.device)]
    for b in range(0, d, 32):
        part = x[:, b:b + 32].double()
        top = part.abs().max(-1, keepdim=True).values
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -149))) - 2
        # log2 rounds up next to a power of two
        e = torch.where(torch.exp2(e + 2) > top, e - 1, e).clamp(-127, 127)
        scale = torch.exp2(e)
        near = ((part.abs() / scale)[..., None] - table).abs().min(-1).indices
        out[:, b:b + 32] = torch.sign(part) * table[near] * scale
    return out


def _exact_sample(s, case):
    B, M, V = s["logits"].shape
    tokens = torch.full((B, M), -1, dtype=torch.int64)
    probs = torch.zeros(B, M, dtype=torch.float64)
    limits = list(zip(*(s[n].tolist() for n in ("temperature", "top_k", "top_p", "min_p"))))
    us = s["uniforms"].tolist()
    for b in range(B):
        T, k, p, m = limits[b]
        for j in range(M):
            x = s["logits"][b, j].double()
            top, at = torch.max(x, 0)
            if T < 1e-5:
                if top > -math.inf:
                    tokens[b, j], probs[b, j] = torch.nonzero(x == top)[0, 0].item(), 1.0
                continue
            q = torch.softmax(x / T, 0)
            if not torch.isfinite(top):
                continue
            # those that can be kept, in the order of falling probability
            live = torch.nonzero((x > -math.inf) & (q >= m * q[at]))[:, 0]
            live = live[torch.sort(x[live], descending=True, stable=True).indices]
            if k > 0:
                live = live[:k]
            share = q[live] / q[live].sum()
            if p < 1:
                before = share.cumsum(0).roll(1)
                before[0] = -1.0
                live = live[before < p]
            live = live.sort().values
            share = q[live] / q[live].sum()
            i = int((share.cumsum(0) <= us[b][j]).sum().clamp(max=live.numel() - 1))
            tokens[b, j], probs[b, j] = live[i].item(), share[i].item()
    return {"tokens": tokens.cuda(), "probs": probs.cuda()}


def _exact_distill(s):
    tau, (B, M, V) = s["tau"], s["logits"].shape
    loss = torch.zeros(B, M, device="cuda", dtype=torch.float64)
    grad = torch.zeros(B, M, V, device="cuda", dtype=torch.float64)
    for b in range(B):
        x = s["logits"][b].double() / tau
        logp = x - torch.logsumexp(x, -1, keepdim=True)
        t = s["teacher_logits"][b].double() / tau
        valid = (s["teacher_ids"][b] >= 0) & (s["teacher_ids"][b] < V)
        for j in range(M):
            ids = s["teacher_ids"][b, j][valid[j]]
            if ids.numel() == 0:
                continue
            logq = torch.log_softmax(t[j][valid[j]], 0)
            loss[b, j] = tau ** 2 * torch.sum(torch.exp(logq) * (logq - logp[j][ids]))
            grad[b, j] = torch.exp(logp[j])
            grad[b, j].index_put_((ids,), -torch.exp(logq), accumulate=True)
            grad[b, j] *= s["grad_loss"][b, j].double() * tau
    return {"loss": loss, "grad": grad}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        out = torch.empty(case["rows"], case["d"], device="cuda", dtype=torch.float64)
        for r in range(0, case["rows"], 32768):
            out[r:r + 32768] = _exact_blocks(s["x"][r:r + 32768])
        return {"values": out}
    if op == "head":
        x = _exact_blocks(s["x"])
        d, V = case["d"], case["V"]
        y = torch.empty(case["rows"], V, device="cuda", dtype=torch.float64)
        for v in range(0, V, 16384):
            c = s["codes"][v:v + 16384].long()
            c = torch.stack([c & 15, c >> 4], -1).view(c.shape[0], -1)[:, :d]
            mag = c & 7  # 0, 1/2, then (1 + bit 0 / 2) 2^(bits 1, 2 - 1)
            w = torch.where(mag < 2, mag * 0.5, (1 + (mag & 1) * 0.5) * torch.exp2((mag >> 1).double() - 1))
            w = torch.where(c > 7, -w, w)
            e = s["scales"][v:v + 16384].double().repeat_interleave(32, 1)[:, :d]
            y[:, v:v + 16384] = x @ (w * torch.exp2(e - 127)).t().contiguous()
        return {"logits": y}
    if op == "sample":
        return _exact_sample(s, case)
    return _exact_distill(s)
