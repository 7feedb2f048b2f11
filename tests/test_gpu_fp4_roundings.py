"""The 4-bit quantiser's roundings: every bf16 number that a scale admits, and
the ties between codes with their neighbours in fp32 and bf16, at scales of both
ends and the middle."""
import numpy as np
import pytest
import torch

import rank_markov_draft_amd as rmd
from tests import blocks_reference as ref

pytestmark = pytest.mark.gpu

BYTES = [0, 1, 2, 3, 64, 126, 127, 128, 200, 251, 252]


def _check(values, byte, dtype):
    """Blocks of 31 of the values behind a number that has the block's scale."""
    top = np.ldexp(4.0, byte - 127)
    v = np.concatenate([values, np.zeros(-values.size % 31, np.float32)]).reshape(-1, 31)
    x = torch.from_numpy(np.concatenate([np.full((v.shape[0], 1), top, np.float32), v], axis=1).astype(np.float32))
    assert torch.equal(x.to(dtype).float(), x)
    codes, scales = rmd.quantize_blocks_fp4(x.to(dtype).cuda())
    wc, ws = ref.quantize(x.numpy())
    assert (ws[:, 0] == byte).all() and np.array_equal(scales.cpu().numpy(), ws)
    got = ref.unpack(codes.cpu().numpy())
    off = np.where(got == 8, 0, got) != np.where(wc == 8, 0, wc)  # both zeros stand for zero
    assert not off[:, 32:].any()
    assert not off.any(), f"byte {byte}: {x.numpy()[off[:, :32]][:5]} gave {got[off][:5]}, want {wc[off][:5]}"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("byte", BYTES)
def test_every_bf16_number(native, byte, dtype):
    v = (np.arange(1 << 16, dtype=np.uint32) << 16).view(np.float32)
    with np.errstate(invalid="ignore"):
        _check(v[np.abs(v.astype(np.float64)) < np.ldexp(8.0, byte - 127)], byte, dtype)


@pytest.mark.parametrize("byte", BYTES)
def test_ties_and_their_neighbours(native, byte):
    at = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0]
    v = np.ldexp(np.array(at), byte - 127).astype(np.float32)
    near = [v]
    up = down = v
    for _ in range(4):
        up, down = np.nextafter(up, np.float32(np.inf)), np.nextafter(down, np.float32(0))
        near += [up, down]
    near = np.concatenate(near)
    _check(np.concatenate([near, -near]), byte, torch.float32)
    # and random fp32 numbers between them, evenly and over all magnitudes
    g = np.random.default_rng(byte)
    v = np.concatenate([g.uniform(-8, 8, 100000), g.choice([-1, 1], 100000) * 8 * np.exp2(-30 * g.random(100000))])
    v = np.ldexp(v, byte - 127).astype(np.float32)
    _check(v[np.abs(v.astype(np.float64)) < np.ldexp(8.0, byte - 127)], byte, torch.float32)
