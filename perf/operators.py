"""What is measured of the int8 vocabulary head and of the logit rules
(penalties for repeated tokens, biases, grammar masks).

Each case names an operator (``op``) and its sizes.  With ``own`` false,
``run`` computes the operators with elementary torch operations in 32 bits;
with ``own`` true it makes the calls of the framework.
"""
import math

import torch

own = False

F32, BF16 = "float32", "bfloat16"


def listed():
    return [
        # rows quantised ahead of the head: one decode batch of hidden states,
        # and the head's own weight when a server loads it
        dict(name="quantize hidden 64", op="quantize", rows=64, d=5120, dtype=BF16),
        dict(name="quantize head", op="quantize", rows=129280, d=5120, dtype=BF16),
        # the head: a single token, a verified block of 64 requests, a ragged
        # batch on a small odd vocabulary, a training-sized batch of blocks
        dict(name="head 1 token", op="head", rows=1, d=5120, V=129280, dtype=BF16, out=F32),
        dict(name="head 64x5", op="head", rows=320, d=5120, V=129280, dtype=BF16, out=F32),
        dict(name="head odd", op="head", rows=37, d=2056, V=32003, dtype=F32, out=BF16),
        dict(name="head 512x5", op="head", rows=2560, d=5120, V=129280, dtype=BF16, out=BF16),
        # the rules on given logits: one request, one position; a large
        # teacher-forced batch with every rule on
        dict(name="process 1 token", op="process", B=1, M=1, V=129280, L=1000, dtype=BF16, bias="none", mask="none"),
        dict(name="process 256x8", op="process", B=256, M=8, V=151936, L=2048, dtype=F32, bias="shared", mask="each"),
        # their gradient: the 320-row batch, and odd sizes
        dict(name="backward 64x5", op="backward", B=64, M=5, V=129280, L=1024, dtype=BF16, mask="each"),
        dict(name="backward odd", op="backward", B=9, M=7, V=50257, L=333, dtype=F32, mask="row"),
        # left to right: the 64-request block greedily, and one request at a
        # temperature on an odd vocabulary
        dict(name="sample greedy 64x5", op="sample", B=64, M=5, V=129280, r=256, L=1024, dtype=BF16, wdtype=BF16,
             T=0.0, bias="none", mask="each"),
        dict(name="sample 1x4", op="sample", B=1, M=4, V=50257, r=64, L=700, dtype=F32, wdtype=F32, T=0.7,
             bias="row", mask="row"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "head", "head", "process", "backward", "sample"])
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
    c = dict(op=op, B=_spread(rng, 1, 64 if op == "sample" else 200), M=rng.randint(1, 8), V=V,
             L=_spread(rng, 1, 4096), dtype=dt, mask=rng.choice(["none", "row", "each"]))
    if op != "backward":
        c["bias"] = rng.choice(["none", "shared", "row"])
    if op == "sample":
        c.update(r=rng.choice([16, 50, 64, 128, 256]), wdtype=rng.choice([F32, BF16]), T=rng.choice([0.0, 0.7]))
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
        s["x"] = normal(case["rows"], case["d"]).to(_dtype(case["dtype"]))
        if op == "head":
            V, d = case["V"], case["d"]
            s["head_q"] = (normal(V, d) * 32).round_().clamp_(-127, 127).to(torch.int8)
            s["head_scale"] = (0.02 / 32) * (0.5 + uniform(V))
        return s
    B, M, V, L = case["B"], case["M"], case["V"], case["L"]
    s["logits"] = normal(B, M, V).mul_(2.0)
    if op == "sample":  # a drafter's confident position
        s["logits"].scatter_add_(2, (uniform(B, M, 1) * V).long(), torch.full((B, M, 1), 6.0, device="cuda"))
    s["logits"] = s["logits"].to(_dtype(case["dtype"]))
    # text repeats its frequent tokens; the rest of a request's row is padding
    s["history"] = (uniform(B, L).pow_(3) * V).long()
    s["lengths"] = L - (uniform(B) * (L // 2 + 1)).long()
    s["prompt_lengths"] = (uniform(B) * (s["lengths"] + 1)).long()
    s["history"][torch.arange(L, device="cuda")[None] >= s["lengths"][:, None]] = -1
    s["repetition"] = 1.0 + 0.3 * uniform(B)
    s["frequency"] = 0.5 * uniform(B)
    s["presence"] = 0.5 * uniform(B)
    if op != "sample":
        s["token_ids"] = (uniform(B, M).pow_(3) * V).long()
    W = (V + 31) // 32
    s["mask"] = None
    if case["mask"] != "none":
        # half of the rows inside free text (nearly all tokens allowed), half
        # at a structural position (few); the last row of a batch at a dead end
        rows = (B, M) if case["mask"] == "each" else (B, 1)

        def words(n):
            w = torch.randint(-(1 << 31), 1 << 31, (n, *rows, W), device="cuda", generator=g, dtype=torch.int64)
            return w.to(torch.int32)

        a = words(5)
        many, few = a[0], a[0]
        for i in range(1, 5):
            many, few = many | a[i], few & a[i]
        s["mask"] = torch.where((uniform(*rows, 1) < 0.5), many, few)
        if B > 7:
            s["mask"][-1, -1] = 0
    s["bias"] = None
    if case.get("bias", "none") != "none":
        rows = 1 if case["bias"] == "shared" else B
        s["bias"] = torch.where(uniform(rows, V) < 0.01, 4.0 * normal(rows, V), torch.zeros((), device="cuda"))
        s["bias"] = s["bias"][0] if case["bias"] == "shared" else s["bias"]
    if op == "backward":
        s["grad"] = normal(B, M, V).to(s["logits"].dtype)
    if op == "sample":
        s["first"] = (uniform(B) * V).long()
        s["w1"], s["w2"] = ((0.02 * normal(V, case["r"])).to(_dtype(case["wdtype"])) for _ in range(2))
        s["noise_seed"] = seed * 7919 + 12345
    return s


# ------------------------------------------------------------ plain forms
def _quantize(x):
    x = x.float()
    top = x.abs().amax(-1)
    scale = top / torch.full_like(top, 127.0)  # a division by a number would be a product with its reciprocal
    q = torch.where(scale[..., None] > 0, torch.round(x / scale[..., None]), torch.zeros_like(x))
    return q.clamp_(-127, 127), scale


def _head(s):
    q, scale = _quantize(s["x"])
    y = q @ s["head_q"].float().t()
    return y.mul_(scale[:, None] * s["head_scale"][None, :]).to(_dtype(s["out"]))


def _history_counts(s, V):
    """Times each token stands among the outputs, and whether it stands anywhere, [B, V]."""
    ids, at = s["history"], torch.arange(s["history"].shape[1], device="cuda")[None]
    ok = (at < s["lengths"][:, None]) & (ids >= 0) & (ids < V)
    safe = torch.where(ok, ids, torch.zeros_like(ids))
    count = torch.zeros(ids.shape[0], V, device="cuda")
    output = ok & (at >= s["prompt_lengths"][:, None])
    count.scatter_add_(1, safe, output.float())
    seen = torch.zeros(ids.shape[0], V, device="cuda")
    seen.scatter_add_(1, safe, ok.float())
    return count, seen


def _block_counts(s, V):
    """The same for every position of the block, [B, M, V]: the tokens of the block before it count too."""
    count, seen = _history_counts(s, V)
    B, M = s["token_ids"].shape
    own_ids = torch.zeros(B, M, V, device="cuda")
    if M > 1:
        own_ids[:, 1:].scatter_(2, s["token_ids"][:, 1:, None], 1.0)
    own_ids = own_ids.cumsum(1)
    return own_ids + count[:, None], own_ids + seen[:, None] > 0


def _allowed(mask, V):
    at = torch.arange(V, device="cuda")
    return (mask[..., at // 32] >> (at % 32)) & 1 != 0


def _rules(x, count, seen, rep, freq, pres, bias, allowed):
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = torch.where(count > 0, x - (freq * count + pres), x)
    if bias is not None:
        x = x + bias
    if allowed is not None:
        x = torch.where(allowed, x, torch.full_like(x, -math.inf))
    return x


def _process(s):
    x = s["logits"].float()
    V = x.shape[-1]
    count, seen = _block_counts(s, V)
    rep, freq, pres = (s[k][:, None, None] for k in ("repetition", "frequency", "presence"))
    bias = s["bias"] if s["bias"] is None or s["bias"].dim() == 1 else s["bias"][:, None]
    allowed = None if s["mask"] is None else _allowed(s["mask"], V)
    return _rules(x, count, seen, rep, freq, pres, bias, allowed).to(s["logits"].dtype)


def _backward(s):
    x, g = s["logits"].float(), s["grad"].float()
    V = x.shape[-1]
    _, seen = _block_counts(s, V)
    rep = s["repetition"][:, None, None]
    g = torch.where(seen, torch.where(x > 0, g / rep, g * rep), g)
    if s["mask"] is not None:
        g = torch.where(_allowed(s["mask"], V), g, torch.zeros_like(g))
    return g.to(s["grad"].dtype)


def _mul32(a, b):
    """High and low words of the product of a 32-bit constant and 32-bit values held in int64."""
    lo, hi = a * (b & 0xFFFF), a * (b >> 16)
    mid = hi + (lo >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (lo & 0xFFFF)


def _gumbel(seed, B, k, V):
    """Base-2 Gumbel noise of position k: Philox4x32-10 (Salmon et al., SC'11) at counter (v / 4, k, b, 0)."""
    n = (V + 3) // 4
    c = [torch.arange(n, device="cuda")[None].expand(B, n), torch.full((B, n), k, device="cuda"),
         torch.arange(B, device="cuda")[:, None].expand(B, n), torch.zeros(B, n, device="cuda", dtype=torch.int64)]
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        h0, l0 = _mul32(0xD2511F53, c[0])
        h2, l2 = _mul32(0xCD9E8D57, c[2])
        c = [h2 ^ c[1] ^ k0, l2, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    u = (2 * (torch.stack(c, -1).reshape(B, 4 * n)[:, :V] >> 9) + 1).double() * 2.0 ** -24
    return -torch.log2(-torch.log2(u))


def _choose(c, T, seed, k):
    """First of the largest scores of each row; -1 where nothing is above -inf."""
    score = c
    if T >= 1e-5:
        kappa = torch.tensor(1.4426950408889634 / T, dtype=torch.float32).double()
        score = (c.double() * kappa + _gumbel(seed, c.shape[0], k, c.shape[1]).float().double()).float()
    top = score.amax(-1, keepdim=True)
    at = torch.arange(c.shape[1], device="cuda")
    first = torch.where(score == top, at, c.shape[1]).amin(-1)
    return torch.where(top[:, 0] > -math.inf, first, -1)


def _sample(s):
    B, M, V = s["logits"].shape
    count, seen = _history_counts(s, V)
    rep, freq, pres = (s[k][:, None] for k in ("repetition", "frequency", "presence"))
    w1, w2 = s["w1"].float(), s["w2"].float().t()
    prev, tokens, rows = s["first"], [], []
    for k in range(M):
        valid = ((prev >= 0) & (prev < V))[:, None]
        bias = (w1[prev.clamp(0, V - 1)] @ w2).to(s["w2"].dtype).float()
        x = (s["logits"][:, k].float() + torch.where(valid, bias, 0.0).to(s["logits"].dtype).float())
        x = x.to(s["logits"].dtype).float()
        mask = None if s["mask"] is None else _allowed(s["mask"][:, k if s["mask"].shape[1] > 1 else 0], V)
        c = _rules(x, count, seen > 0, rep, freq, pres, s["bias"], mask).to(s["logits"].dtype)
        prev = _choose(c.float(), s["T"], s["noise_seed"], k)
        hit = (prev >= 0).float()[:, None]
        count.scatter_add_(1, prev.clamp(min=0)[:, None], hit)
        seen.scatter_add_(1, prev.clamp(min=0)[:, None], hit)
        tokens.append(prev)
        rows.append(c)
    return {"tokens": torch.stack(tokens, 1), "logits": torch.stack(rows, 1)}


# ------------------------------------------------------------ one pass
def _own(s):
    import rank_markov_draft_amd as rmd

    op = s["op"]
    if op == "quantize":
        q, scale = rmd.quantize_rows(s["x"])
        return {"q": q, "scale": scale}
    if op == "head":
        return {"logits": rmd.lm_head_logits_int8(s["x"], s["head_q"], s["head_scale"], out_dtype=_dtype(s["out"]))}
    seen = dict(history=s["history"], lengths=s["lengths"], prompt_lengths=s["prompt_lengths"],
                repetition_penalty=s["repetition"], token_mask=s["mask"])
    if op == "backward":
        return {"grad": rmd.process_block_logits_backward(s["grad"], s["logits"], token_ids=s["token_ids"], **seen)}
    seen.update(frequency_penalty=s["frequency"], presence_penalty=s["presence"], logit_bias=s["bias"])
    if op == "process":
        return {"logits": rmd.process_block_logits(s["logits"], token_ids=s["token_ids"], **seen)}
    if "workspace" not in s:  # a server keeps it beside its weights
        B, M, V = s["logits"].shape
        s["workspace"] = rmd.Workspace(B, M, V, s["r"], sample=True, processed=True)
    tokens, logits = rmd.sample_block_tokens_processed(s["logits"], s["first"], s["w1"], s["w2"], s["T"],
                                                       seed=s["noise_seed"], workspace=s["workspace"], **seen)
    return {"tokens": tokens, "logits": logits}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "quantize":
        q, scale = _quantize(state["x"])
        return {"q": q.to(torch.int8), "scale": scale}
    if op == "head":
        return {"logits": _head(state)}
    if op == "process":
        return {"logits": _process(state)}
    if op == "backward":
        return {"grad": _backward(state)}
    return _sample(state)


def work(case):
    size = {F32: 4, BF16: 2}
    op, es = case["op"], size[case["dtype"]]
    if op == "quantize":
        n = case["rows"] * case["d"]
        return {"bytes": n * (es + 1) + 4 * case["rows"], "flops": 0}
    if op == "head":
        rows, d, V = case["rows"], case["d"], case["V"]
        return {"bytes": V * (d + 4) + rows * d * es + rows * V * size[case["out"]], "flops": 2 * rows * d * V}
    B, M, V = case["B"], case["M"], case["V"]
    n = B * M * V
    total = 2 * n * es + 8 * B * (case["L"] * 3 // 4)
    total += {"none": 0, "row": B * V // 8, "each": n // 8}[case["mask"]]
    total += {"none": 0, "shared": 4 * V, "row": 4 * B * V}[case.get("bias", "none")]
    if op == "sample":
        total += size[case["wdtype"]] * case["r"] * (V + B * M)
        return {"bytes": total, "flops": 2 * n * case["r"]}
    return {"bytes": total, "flops": 0}


# ------------------------------------------------------------ in 64 bits
def _exact_q(x):
    """The scale and the quotients are fp32 by the operator's definition: rounded there, everything else in 64 bits."""
    x = x.double()
    scale = (x.abs().max(-1).values / 127.0).float().double()
    quot = (x / scale.clamp(min=1e-300)[:, None]).float().double()
    return torch.where(scale[:, None] > 0, quot.round().clamp(-127, 127), 0.0), scale


def _exact_tables(s, V, blocks):
    """Counts by sorting the ids of each request, [B, V] pairs of tables for each number of the block's tokens."""
    ids = s["history"].cpu()
    count = torch.zeros(ids.shape[0], V, dtype=torch.float64)
    seen = torch.zeros(ids.shape[0], V, dtype=torch.bool)
    for b in range(ids.shape[0]):
        n, p = int(s["lengths"][b]), int(s["prompt_lengths"][b])
        u, c = torch.unique(ids[b, p:n], return_counts=True)
        count[b, u] = c.double()
        seen[b, torch.unique(ids[b, :n])] = True
    count, seen = count.cuda(), seen.cuda()
    yield count, seen
    for k in range(1, blocks):
        t = s["token_ids"][:, k]
        for b in range(t.shape[0]):
            count[b, t[b]] += 1
            seen[b, t[b]] = True
        yield count, seen


def _exact_bits(words, V):
    """Truth values of packed words, by bytes of eight."""
    w = words.contiguous().view(torch.uint8)
    bits = torch.stack([(w >> i) & 1 for i in range(8)], -1).reshape(*words.shape[:-1], -1)
    return bits[..., :V].bool()


def _exact_rules(x, count, seen, s, allowed):
    rep, freq, pres = (s[k].double()[:, None] for k in ("repetition", "frequency", "presence"))
    divided = seen & (x > 0)
    x = x / torch.where(divided, rep, 1.0) * torch.where(seen & ~divided, rep, 1.0)
    x = x - (count * freq + (count > 0) * pres)
    if s["bias"] is not None:
        x = x + s["bias"].double()
    return x if allowed is None else x.masked_fill(~allowed, -math.inf)


def _exact_choice(c, T, seed, k):
    """The first column in the order of falling scores; -1 if its score is -inf."""
    if T >= 1e-5:
        c = c * (math.log2(math.e) / T) + _gumbel(seed, c.shape[0], k, c.shape[1])
    score, column = torch.sort(c, dim=-1, descending=True, stable=True)
    return torch.where(torch.isinf(score[:, 0]) & (score[:, 0] < 0), -1, column[:, 0])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        q, scale = _exact_q(s["x"])
        return {"q": q.to(torch.int8), "scale": scale}
    if op == "head":
        q, scale = _exact_q(s["x"])
        y = torch.empty(case["rows"], case["V"], device="cuda", dtype=torch.float64)
        for v in range(0, case["V"], 16384):
            part = slice(v, min(case["V"], v + 16384))
            y[:, part] = q @ s["head_q"][part].double().t().contiguous()
            y[:, part] *= scale[:, None] * s["head_scale"][part].double()[None, :]
        return {"logits": y}
    B, M, V = case["B"], case["M"], case["V"]
    if op in ("process", "backward"):
        y = torch.empty(B, M, V, device="cuda", dtype=torch.float64)
        for k, (count, seen) in enumerate(_exact_tables(s, V, M)):
            allowed = None if s["mask"] is None else _exact_bits(s["mask"][:, k if s["mask"].shape[1] > 1 else 0], V)
            x = s["logits"][:, k].double()
            if op == "process":
                y[:, k] = _exact_rules(x, count, seen, s, allowed)
            else:
                rep = s["repetition"].double()[:, None]
                slope = torch.where(x > 0, 1.0 / rep, rep)
                y[:, k] = s["grad"][:, k].double() * torch.where(seen, slope, 1.0)
                if allowed is not None:
                    y[:, k] *= allowed
        return {"logits" if op == "process" else "grad": y}
    # left to right: the roundings of the corrected and the processed logits
    # decide the tokens, so they belong to the definition
    L, Wt = s["logits"].dtype, s["w2"].dtype
    count, seen = next(_exact_tables(s, V, 1))
    prev, tokens = s["first"], []
    y = torch.empty(B, M, V, device="cuda", dtype=torch.float64)
    w2 = s["w2"].double().t().contiguous()
    for k in range(M):
        ok = (prev >= 0) & (prev < V)
        e = torch.where(ok[:, None], s["w1"][prev.clamp(0, V - 1)].double(), 0.0)
        x = s["logits"][:, k].double() + (e @ w2).to(Wt).double().to(L).double()
        allowed = None if s["mask"] is None else _exact_bits(s["mask"][:, k if s["mask"].shape[1] > 1 else 0], V)
        y[:, k] = _exact_rules(x.to(L).double(), count, seen, s, allowed)
        prev = _exact_choice(y[:, k].to(L).double(), case["T"], s["noise_seed"], k)
        for b in range(B):
            if prev[b] >= 0:
                count[b, prev[b]] += 1
                seen[b, prev[b]] = True
        tokens.append(prev)
    return {"tokens": torch.stack(tokens, 1), "logits": y}
