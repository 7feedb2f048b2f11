"""Host-side refusals of the 4-bit head, of sampling under limits and of the
distillation loss: by the C ABI (nothing reaches a kernel) and by the Python
binding (before any library call).  No GPU."""
import ctypes

import pytest
import torch

import rank_markov_draft_amd as rmd
from rank_markov_draft_amd import _lib

MB = 1 << 24
A = [ctypes.c_void_p(MB * (i + 1)) for i in range(16)]   # distinct addresses, never dereferenced
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3
FULL = 2 ** 64 - 1


@pytest.fixture(scope="module")
def L():
    return _lib.load()


def at(p, off):
    return ctypes.c_void_p(p.value + off)


def _data(L):
    return L.dspark_markov_workspace_bytes(1, 1, 8, 8, 0) - 16384


# ------------------------------------------------------------ 4-bit blocks
def test_quantize_refusals(L):
    def q(x=A[0], dt=1, rows=4, d=40, c=A[1], s=A[2]):
        return L.dspark_markov_quantize_fp4(x, dt, rows, d, c, s, None)
    for kw in (dict(dt=5), dict(rows=-1), dict(d=-1), dict(x=None), dict(c=None), dict(s=None), dict(rows=2 ** 62),
               dict(rows=2 ** 57), dict(c=at(A[1], 8)), dict(s=at(A[2], 2)), dict(c=at(A[0], 16)), dict(s=at(A[0], 16)),
               dict(s=at(A[1], 252))):
        assert q(**kw) == INVALID, kw
    assert q(d=2 ** 20 + 1) == UNSUPPORTED and b"1048576" in L.dspark_markov_last_error()
    assert q(rows=0, x=None, c=None, s=None) == OK and q(d=0, x=None, c=None, s=None) == OK


def test_dequantize_refusals(L):
    def q(c=A[1], s=A[2], rows=4, d=40, x=A[0], dt=0):
        return L.dspark_markov_dequantize_fp4(c, s, rows, d, x, dt, None)
    for kw in (dict(dt=-1), dict(rows=-1), dict(d=-1), dict(x=None), dict(c=None), dict(s=None), dict(rows=2 ** 62),
               dict(c=at(A[1], 4)), dict(s=at(A[2], 1)), dict(x=at(A[1], 16)), dict(x=at(A[2], 8))):
        assert q(**kw) == INVALID, kw
    assert q(d=2 ** 20 + 1) == UNSUPPORTED
    assert q(rows=0, x=None, c=None, s=None) == OK and q(d=0, x=None, c=None, s=None) == OK


def test_head_workspace_and_refusals(L):
    data = _data(L)
    size = L.dspark_markov_lm_head_fp4_workspace_bytes
    assert size(4, 5, 100) == data + 20 * 128 + 256       # one chunk of codes a row, and its 8 scale bytes
    assert size(4, 5, 300) == data + 20 * 256 + 512
    assert size(2 ** 40, 2 ** 40, 100) == FULL and size(2 ** 60, 1, 2 ** 20) == FULL and size(-1, 5, 100) == data

    def h(hid=A[0], hdt=1, d=64, c=A[1], s=A[2], B=2, M=3, V=40, out=A[3], odt=0, ws=A[4], n=1 << 23):
        return L.dspark_markov_lm_head_fp4(hid, hdt, d, c, s, B, M, V, out, odt, ws, n, None)
    for kw in (dict(hdt=9), dict(odt=2), dict(d=0), dict(d=-3), dict(B=-1), dict(M=-1), dict(V=-1), dict(hid=None),
               dict(c=None), dict(s=None), dict(out=None), dict(B=2 ** 40, M=2 ** 40), dict(V=2 ** 58, B=1, M=1),
               dict(out=at(A[0], 8)), dict(out=at(A[1], 100)), dict(out=at(A[2], 4)), dict(c=at(A[1], 8)),
               dict(s=at(A[2], 2)), dict(ws=at(A[4], 8)), dict(ws=at(A[0], -data)), dict(ws=at(A[3], -data)),
               dict(ws=at(A[1], 16 - data))):
        assert h(**kw) == INVALID, kw
    assert h(d=2 ** 20 + 1) == UNSUPPORTED and b"1048576" in L.dspark_markov_last_error()
    assert h(V=2 ** 31, B=1, M=1) == UNSUPPORTED
    assert h(ws=None) == SMALL and h(n=data) == SMALL
    assert h(B=0) == OK and h(V=0) == OK and h(M=0, hid=None) == OK


# ------------------------------------------------------------ sampling under limits
def test_sample_workspace_and_refusals(L):
    data = _data(L)
    size = L.dspark_markov_sample_filtered_workspace_bytes
    assert size(2, 3, 1000) == data + 512 + 256           # 8 groups a row: 8 and 4 bytes each
    assert size(2 ** 40, 2 ** 40, 8) == FULL and size(2 ** 32, 2 ** 20, 2 ** 40) == FULL and size(1, -1, 8) == data

    def lim(**kw):
        r = _lib.TokenLimits()
        r.all_temperature, r.all_top_p = 1.0, 1.0
        for k, v in kw.items():
            setattr(r, k, v.value)
        return r

    def f(x=A[0], dt=0, u=A[1], l=lim(), B=2, M=3, V=40, t=A[2], p=A[3], ws=A[4], n=1 << 23):
        return L.dspark_markov_sample_filtered(x, dt, u, l, B, M, V, t, p, ws, n, None)
    for kw in (dict(dt=7), dict(B=-1), dict(M=-1), dict(V=-1), dict(V=0), dict(x=None), dict(u=None), dict(l=None),
               dict(t=None), dict(p=None), dict(B=2 ** 40, M=2 ** 40), dict(B=2 ** 60, V=1, M=1), dict(t=at(A[0], 8)),
               dict(p=at(A[0], 8)), dict(t=at(A[1], 8)), dict(p=at(A[1], 20)), dict(p=at(A[2], 40)),
               dict(l=lim(temperature=A[2])), dict(l=lim(top_k=A[3])), dict(l=lim(top_p=at(A[2], 44))),
               dict(l=lim(min_p=A[3])), dict(ws=at(A[4], 8)), dict(ws=at(A[0], -data)), dict(ws=at(A[2], -data)),
               dict(ws=at(A[3], 16 - data))):
        assert f(**kw) == INVALID, kw
    assert f(V=2 ** 30 + 1) == UNSUPPORTED
    assert f(ws=None) == SMALL and f(n=data) == SMALL
    assert f(B=0) == OK and f(M=0, x=None, t=None) == OK


# ------------------------------------------------------------ distillation
def test_distill_workspace_and_refusals(L):
    data = _data(L)
    size = L.dspark_markov_distill_workspace_bytes
    assert size(1, 1, 8192) == data + 256 and size(1, 1, 8192 * 100) == data + 1024 and size(4096, 1, 10 ** 6) == data + 6144 * 8
    assert size(2 ** 40, 2 ** 40, 8) == FULL and size(1, 1, 2 ** 63 - 1) == data + 2048 * 8
    assert size(2 ** 62, 1, 8) == FULL and size(2 ** 63 - 1, 1, 2 ** 40) == FULL
    # a workspace serves every smaller call
    for V in (1, 9000, 129280):
        last = 0
        for rows in (1, 2, 7, 100, 1023, 1024, 2047, 2048, 2049, 5000):
            assert size(rows, 1, V) >= last
            last = size(rows, 1, V)

    def f(x=A[0], dt=0, ids=A[1], t=A[2], tdt=0, B=2, M=3, V=40, K=5, T=1.0, loss=A[3], st=A[4], ws=A[5], n=1 << 23):
        return L.dspark_markov_distill_block(x, dt, ids, t, tdt, B, M, V, K, T, loss, st, ws, n, None)
    bad = [dict(dt=3), dict(tdt=-1), dict(B=-1), dict(M=-1), dict(V=-1), dict(V=0), dict(K=-1), dict(x=None), dict(ids=None),
           dict(t=None), dict(T=0.0), dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-40), dict(T=1e40),
           dict(B=2 ** 40, M=2 ** 40), dict(B=2 ** 40, M=2 ** 20, V=8)]
    for kw in bad + [dict(loss=None), dict(st=None), dict(loss=at(A[0], 4)), dict(loss=at(A[1], 8)), dict(st=at(A[2], 4)),
                     dict(st=at(A[0], 4)), dict(st=at(A[3], 16)), dict(ws=at(A[5], 8)), dict(ws=at(A[0], -data)),
                     dict(ws=at(A[3], -data)), dict(ws=at(A[4], 16 - data))]:
        assert f(**kw) == INVALID, kw
    assert f(V=2 ** 30 + 1) == UNSUPPORTED and f(K=1025) == UNSUPPORTED
    assert f(ws=None) == SMALL and f(n=data) == SMALL
    assert f(B=0) == OK and f(M=0, x=None, loss=None) == OK

    def b(g=A[6], x=A[0], dt=0, ids=A[1], t=A[2], tdt=0, st=A[4], B=2, M=3, V=40, K=5, T=1.0, out=A[7]):
        return L.dspark_markov_distill_block_backward(g, x, dt, ids, t, tdt, st, B, M, V, K, T, out, None)
    for kw in bad + [dict(g=None), dict(st=None), dict(out=None), dict(out=at(A[0], 4)), dict(out=at(A[1], 8)),
                     dict(out=A[2]), dict(out=A[4]), dict(out=at(A[6], 4))]:
        assert b(**kw) == INVALID, kw
    assert b(V=2 ** 30 + 1) == UNSUPPORTED and b(K=1025) == UNSUPPORTED
    assert b(B=0) == OK and b(M=0, x=None, out=None) == OK


# ------------------------------------------------------------ binding
def _cpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_host_tensors():
    u8, ids = torch.uint8, _cpu(2, 3, 4, dtype=torch.int64)
    x = _cpu(2, 3, 40)
    for call in (lambda: rmd.quantize_blocks_fp4(x), lambda: rmd.dequantize_blocks_fp4(_cpu(2, 64, dtype=u8), _cpu(2, 4, dtype=u8), 40),
                 lambda: rmd.lm_head_logits_fp4(x, _cpu(9, 64, dtype=u8), _cpu(9, 4, dtype=u8)),
                 lambda: rmd.sample_block_filtered(x, _cpu(2, 3)), lambda: rmd.distill_block_loss(x, ids, _cpu(2, 3, 4)),
                 lambda: rmd.distill_block_loss_backward(_cpu(2, 3), x, ids, _cpu(2, 3, 4), _cpu(2, 3, 4))):
        with pytest.raises(ValueError, match="runs on a GPU"):
            call()


def test_binding_refuses_shapes_and_types():
    u8, i64 = torch.uint8, torch.int64
    x, ids, t = _cpu(2, 3, 40), _cpu(2, 3, 4, dtype=i64), _cpu(2, 3, 4)
    codes, scales = _cpu(9, 64, dtype=u8), _cpu(9, 4, dtype=u8)
    for call, match in (
            (lambda: rmd.quantize_blocks_fp4(torch.zeros(())), r"\[\.\.\., d\]"),
            (lambda: rmd.dequantize_blocks_fp4(codes, scales, 200), "codes must be uint8"),
            (lambda: rmd.dequantize_blocks_fp4(codes, scales, -1), "codes must be uint8"),
            (lambda: rmd.dequantize_blocks_fp4(codes.to(torch.int8), scales, 100), "codes must be uint8"),
            (lambda: rmd.dequantize_blocks_fp4(codes, scales[:, :3], 100), "scales must be uint8"),
            (lambda: rmd.lm_head_logits_fp4(x, codes[:, :32], scales), "head_codes must be uint8"),
            (lambda: rmd.lm_head_logits_fp4(x, codes.to(torch.int8), scales), "head_codes must be uint8"),
            (lambda: rmd.lm_head_logits_fp4(x, codes, scales[:8]), "head_scales must be uint8"),
            (lambda: rmd.sample_block_filtered(x[0], _cpu(2, 3)), "must be"),
            (lambda: rmd.sample_block_filtered(x, _cpu(2, 2)), "uniforms must be"),
            (lambda: rmd.sample_block_filtered(x, _cpu(2, 3, dtype=i64)), "uniforms must be"),
            (lambda: rmd.sample_block_filtered(x, _cpu(2, 3), _cpu(3)), r"temperature must be a number or \[2\]"),
            (lambda: rmd.sample_block_filtered(x, _cpu(2, 3), top_p=_cpu(2, 3)), r"top_p must be a number or \[2\]"),
            (lambda: rmd.sample_block_filtered(x, _cpu(2, 3), top_k=2 ** 64 + 5), "64 bits"),
            (lambda: rmd.distill_block_loss(x, ids[:1], t), "teacher_ids must be"),
            (lambda: rmd.distill_block_loss(x, t, t), "teacher_ids must be"),
            (lambda: rmd.distill_block_loss(x, ids, t[..., :3]), "teacher_logits must be"),
            (lambda: rmd.distill_block_loss_backward(_cpu(2, 2), x, ids, t, _cpu(2, 3, 4)), "grad_loss must be"),
            (lambda: rmd.distill_block_loss_backward(_cpu(2, 3), x, ids, t, _cpu(2, 3, 3)), "stats must be"),
            (lambda: rmd.distill_block_loss_backward(_cpu(2, 3), x, ids, t, _cpu(2, 3, 4).double()), "stats must be")):
        with pytest.raises(ValueError, match=match):
            call()
    for call in (lambda: rmd.sample_block_filtered(x, _cpu(2, 3), top_k=_cpu(2)),
                 lambda: rmd.sample_block_filtered(x, _cpu(2, 3), _cpu(2, dtype=i64)),
                 lambda: rmd.sample_block_filtered(x, _cpu(2, 3), min_p=_cpu(2, dtype=i64)),
                 lambda: rmd.sample_block_filtered(x, _cpu(2, 3), top_k=3.5)):
        with pytest.raises(TypeError):
            call()
