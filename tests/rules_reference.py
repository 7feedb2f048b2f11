"""The logit rules and the 8-bit head written out in 64 bits (test
infrastructure), with how far a kernel that works in fp32 and rounds once to
its output type may be from them."""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24                                    # half a step of fp32, relative
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133}   # a step of the subnormals


def pack_mask(allowed: np.ndarray) -> np.ndarray:
    """Truth values [..., V] as int32 words of 32 tokens."""
    V = allowed.shape[-1]
    W = (V + 31) // 32
    bits = np.zeros(allowed.shape[:-1] + (W * 32,), np.uint8)
    bits[..., :V] = allowed
    by = np.packbits(bits.reshape(-1, W * 4, 8), axis=-1, bitorder="little")
    return by.reshape(-1).view(np.int32).reshape(allowed.shape[:-1] + (W,))


def counts(history, lengths, prompt_lengths, extra, b, V):
    """(count among outputs [V], seen [V]) of request b; extra: later outputs."""
    count, seen = np.zeros(V), np.zeros(V, bool)
    if history is not None:
        L = history.shape[1]
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        p = 0 if prompt_lengths is None else int(prompt_lengths[b])
        for i in range(n):
            t = int(history[b, i])
            if 0 <= t < V:
                seen[t] = True
                count[t] += i >= p
    for t in extra:
        if 0 <= int(t) < V:
            seen[int(t)] = True
            count[int(t)] += 1
    return count, seen


def rules_row(x, count, seen, rep, freq, pres, bias, allowed):
    """One row in 64 bits and the rounding errors of its fp32 steps (without
    the last rounding to the output type).  rep, freq, pres: numbers or None."""
    x = np.asarray(x, np.float64)
    tol = np.zeros_like(x)

    def rounded(y):
        with np.errstate(invalid="ignore"):
            return U32 * np.where(np.isfinite(y), np.abs(y), 0.0) + 2.0 ** -149

    with np.errstate(invalid="ignore", over="ignore"):
        if rep is not None:
            up = x > 0
            slope = np.where(seen, np.where(up, 1.0 / rep, rep), 1.0)
            x = np.where(seen, np.where(up, x / rep, x * rep), x)
            tol = tol * slope + np.where(seen, rounded(x), 0.0)
        if freq is not None or pres is not None:
            f, p = 0.0 if freq is None else freq, 0.0 if pres is None else pres
            off = np.where(count > 0, f * count + p, 0.0)
            x = x - off
            tol = tol + np.where(count > 0, rounded(f * count) + rounded(off) + rounded(x), 0.0)
        if bias is not None:
            x = x + np.asarray(bias, np.float64)
            tol = tol + rounded(x)
        if allowed is not None:
            x = np.where(allowed, x, -np.inf)
    # errors of errors: the terms above are relative to 2^-24, once more
    return x, tol * (1 + 2.0 ** -20)


def check(got: torch.Tensor, ref: np.ndarray, tol: np.ndarray, what: str):
    """got against 64-bit values: equal where those leave the type's range,
    else within tol and the last rounding."""
    dt = got.dtype
    g = got.detach().cpu().double().numpy().reshape(ref.shape)
    with np.errstate(over="ignore", invalid="ignore"):
        want = torch.from_numpy(np.asarray(ref, np.float64)).to(torch.float32).to(dt).double().numpy()
    special = ~np.isfinite(want)
    same = np.where(np.isnan(want), np.isnan(g), g == want)
    # a value within its error of the type's largest may round to it or past it
    bad = special & ~same
    with np.errstate(invalid="ignore"):
        limit = tol + HALF_STEP[dt] * (np.abs(ref) + tol) + TINY[dt]
        bad |= ~special & ~(np.abs(g - ref) <= limit)
    if bad.any():
        at = tuple(int(i[0]) for i in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; first at {at}: got {g[at]!r}, "
                             f"want {ref[at]!r}")


def quantize(x: np.ndarray):
    """q (as float64) and the fp32 scale (as float64) of rows of fp32 values;
    a division of two fp32 numbers done in 64 bits and rounded is the fp32
    division (53 >= 2 * 24 + 2)."""
    x = np.asarray(x, np.float64)
    scale = (np.abs(x).max(-1, initial=0.0) / 127.0).astype(np.float32).astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        quot = (x / scale[..., None]).astype(np.float32).astype(np.float64)
        ok = (scale > 0) & np.isfinite(scale)
        q = np.where(ok[..., None], np.clip(np.rint(quot), -127, 127), 0.0)
    return q, scale
