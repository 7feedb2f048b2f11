"""Host-side refusals of the 8-bit head and the logit rules: by the C ABI
(nothing reaches a kernel) and by the Python binding (before any library
call).  No GPU."""
import ctypes

import pytest
import torch

import rank_markov_draft_amd as rmd
from rank_markov_draft_amd import _lib

MB = 1 << 24
A = [ctypes.c_void_p(MB * (i + 1)) for i in range(16)]   # distinct addresses, never dereferenced
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    return _lib.load()


def at(p, off):
    return ctypes.c_void_p(p.value + off)


# ------------------------------------------------------------ quantiser
def test_quantize_refusals(L):
    def q(x=A[0], dt=1, rows=4, d=8, q=A[1], s=A[2]):
        return L.dspark_markov_quantize_rows(x, dt, rows, d, q, s, None)
    assert q(dt=5) == INVALID and q(rows=-1) == INVALID and q(d=-1) == INVALID
    assert q(x=None) == INVALID and q(q=None) == INVALID and q(s=None) == INVALID
    assert q(rows=0, x=None, q=None, s=None) == OK
    assert q(rows=2 ** 62, d=8) == INVALID and q(rows=2 ** 31, d=1) == UNSUPPORTED
    assert q(q=at(A[0], 16)) == INVALID                  # integers over the rows
    assert q(s=at(A[0], 60)) == INVALID                  # scales over the rows
    assert q(s=at(A[1], 31)) == INVALID                  # scales over the integers


# ------------------------------------------------------------ head
def test_head_workspace_and_refusals(L):
    data = L.dspark_markov_workspace_bytes(1, 1, 8, 8, 0) - 16384
    assert L.dspark_markov_lm_head_int8_workspace_bytes(4, 5, 100) == data + 20 * 128 + 2304
    assert L.dspark_markov_lm_head_int8_workspace_bytes(2 ** 40, 2 ** 40, 100) == 2 ** 64 - 1
    assert L.dspark_markov_lm_head_int8_workspace_bytes(-1, 5, 100) == data

    def h(hid=A[0], hdt=1, d=64, q=A[1], s=A[2], B=2, M=3, V=40, out=A[3], odt=0, ws=A[4], n=1 << 23):
        return L.dspark_markov_lm_head_int8(hid, hdt, d, q, s, B, M, V, out, odt, ws, n, None)
    for kw in (dict(hdt=9), dict(odt=2), dict(d=0), dict(d=-3), dict(B=-1), dict(M=-1), dict(V=-1), dict(hid=None),
               dict(q=None), dict(s=None), dict(out=None), dict(B=2 ** 40, M=2 ** 40), dict(out=at(A[0], 8)),
               dict(out=at(A[1], 100)), dict(out=at(A[2], 4))):
        assert h(**kw) == INVALID, kw
    assert h(d=131073) == UNSUPPORTED and b"131072" in L.dspark_markov_last_error()
    assert h(V=2 ** 31, B=1, M=1, d=16) == UNSUPPORTED
    assert h(ws=None) == SMALL and h(n=data) == SMALL
    assert h(B=0) == OK and h(V=0) == OK and h(M=0, hid=None) == OK


# ------------------------------------------------------------ rules
def rules(**kw):
    r = _lib.LogitRules()
    for k, v in kw.items():
        setattr(r, k, v.value if isinstance(v, ctypes.c_void_p) else v)
    return r


BAD_RULES = [
    dict(history=A[5], history_len=-1, history_stride=4),
    dict(history=A[5], history_len=5, history_stride=4),             # rows over each other
    dict(history=A[5], history_len=2 ** 62, history_stride=2 ** 62),
    dict(logit_bias=A[5], bias_dtype=4),
    dict(logit_bias=A[5], bias_stride=39),
    dict(logit_bias=A[5], bias_stride=-40),
    dict(token_mask=A[5], mask_stride_b=-2),
    dict(token_mask=A[5], mask_stride_m=-2),
    dict(token_mask=A[5], mask_stride_m=2 ** 62),
]


@pytest.mark.parametrize("kw", BAD_RULES)
def test_bad_rules(L, kw):
    r = rules(**kw)
    assert L.dspark_markov_process_block(A[0], 0, None, r, 2, 3, 40, A[1], None) == INVALID
    assert L.dspark_markov_process_block_backward(A[0], A[2], 0, None, r, 2, 3, 40, A[1], None) == INVALID
    assert L.dspark_markov_sample_block_processed(A[0], 1, A[1], A[2], A[3], 1, r, 2, 3, 40, 8, 0.0, 0, 0, 0, A[4], A[6],
                                                  A[7], 1 << 24, None) == INVALID


def test_process_refusals(L):
    def p(x=A[0], dt=0, ids=A[1], r=rules(), B=2, M=3, V=40, out=A[2]):
        return L.dspark_markov_process_block(x, dt, ids, r, B, M, V, out, None)
    for kw in (dict(x=None), dict(dt=7), dict(r=None), dict(B=-1), dict(M=-2), dict(V=-1), dict(out=None),
               dict(B=2 ** 40, M=2 ** 30), dict(out=at(A[0], 4)), dict(out=at(A[1], 8)),
               dict(r=rules(history=A[2], history_len=4, history_stride=4)), dict(r=rules(token_mask=A[2])),
               dict(r=rules(logit_bias=A[2])), dict(r=rules(repetition_penalty=A[2])),
               dict(r=rules(frequency_penalty=A[2])), dict(r=rules(presence_penalty=A[2])),
               dict(r=rules(history=A[5], history_len=4, history_stride=4, lengths=A[2])),
               dict(r=rules(history=A[5], history_len=4, history_stride=4, prompt_lengths=A[2]))):
        assert p(**kw) == INVALID, kw
    assert p(V=2 ** 30 + 1, B=1, M=1) == UNSUPPORTED
    assert p(B=0) == OK and p(M=0) == OK and p(V=0, x=None) == OK

    def b(g=A[0], x=A[3], out=A[2], r=rules()):
        return L.dspark_markov_process_block_backward(g, x, 1, A[1], r, 2, 3, 40, out, None)
    assert b(g=None) == INVALID and b(x=None) == INVALID and b(out=None) == INVALID and b(r=None) == INVALID
    assert b(out=A[3]) == INVALID                            # the logits are read after their gradient is written
    assert b(out=at(A[0], 2)) == INVALID


def test_sample_processed_refusals(L):
    need = L.dspark_markov_processed_workspace_bytes(2, 3, 40, 8)
    assert need == L.dspark_markov_workspace_bytes(2, 3, 40, 8, 1) + 256 + 768 + 512
    # the step reads the counts of a lane's 16 columns of 64 where any of them
    # exists: up to 51 past the last row's end
    for B, V in ((32, 65), (1, 97), (64, 1), (3, 32065)):
        bits = -(-B * (-(-V // 32)) * 4 // 256) * 256
        base = -(-L.dspark_markov_workspace_bytes(B, 2, V, 8, 1) // 256) * 256
        assert L.dspark_markov_processed_workspace_bytes(B, 2, V, 8) >= base + bits + 4 * (B * V + 51)
    assert L.dspark_markov_processed_workspace_bytes(2 ** 40, 1, 2 ** 40, 8) == 2 ** 64 - 1

    def s(base=A[0], ldt=1, first=A[1], w1=A[2], w2=A[3], wdt=1, r_=rules(), B=2, M=3, V=40, r=8, T=0.0, tok=A[4], out=A[6],
          ws=A[7], n=1 << 24):
        return L.dspark_markov_sample_block_processed(base, ldt, first, w1, w2, wdt, r_, B, M, V, r, T, 0, 0, 0, tok, out, ws,
                                                      n, None)
    for kw in (dict(base=None), dict(first=None), dict(w1=None), dict(w2=None), dict(tok=None), dict(out=None), dict(r_=None),
               dict(ldt=3), dict(wdt=3), dict(B=-1), dict(r=0), dict(V=0), dict(T=float("nan")), dict(out=A[0]),
               dict(out=at(A[2], 2)), dict(tok=at(A[1], 8)), dict(tok=at(A[6], 0)),
               dict(r_=rules(token_mask=A[6])), dict(r_=rules(history=A[4], history_len=2, history_stride=2))):
        assert s(**kw) == INVALID, kw
    assert s(ws=None) == SMALL and s(n=need - 1) == SMALL
    assert s(r=16385) == UNSUPPORTED and s(V=2 ** 30 + 8, r=1) == UNSUPPORTED
    assert s(B=0) == OK and s(M=0) == OK


# ------------------------------------------------------------ binding
def test_binding_refuses_host_tensors():
    x, ids = torch.zeros(2, 3, 40), torch.zeros(2, dtype=torch.int64)
    w = torch.zeros(40, 8)
    for call in (lambda: rmd.quantize_rows(x), lambda: rmd.process_block_logits(x),
                 lambda: rmd.process_block_logits_backward(x, x),
                 lambda: rmd.lm_head_logits_int8(torch.zeros(2, 8), torch.zeros(40, 8, dtype=torch.int8), torch.zeros(40)),
                 lambda: rmd.sample_block_tokens_processed(x, ids, w, w)):
        with pytest.raises(ValueError, match="runs on a GPU"):
            call()


def test_binding_refuses_shapes():
    x = torch.zeros(2, 3, 40)
    with pytest.raises(ValueError, match="head_q"):
        rmd.lm_head_logits_int8(torch.zeros(2, 8), torch.zeros(40, 9, dtype=torch.int8), torch.zeros(40))
    with pytest.raises(ValueError, match="head_q"):
        rmd.lm_head_logits_int8(torch.zeros(2, 8), torch.zeros(40, 8), torch.zeros(40))
    with pytest.raises(ValueError, match="head_scale"):
        rmd.lm_head_logits_int8(torch.zeros(2, 8), torch.zeros(40, 8, dtype=torch.int8), torch.zeros(39))
    with pytest.raises(ValueError, match=r"\[B, M, V\]"):
        rmd.process_block_logits(x[0])
    with pytest.raises(ValueError, match="token_ids"):
        rmd.process_block_logits(x, token_ids=torch.zeros(2, 2, dtype=torch.int64))
    with pytest.raises(ValueError, match="token_ids"):
        rmd.process_block_logits(x, token_ids=torch.zeros(2, 3))
    with pytest.raises(ValueError, match="grad_processed"):
        rmd.process_block_logits_backward(x.to(torch.bfloat16), x)
    with pytest.raises(ValueError, match="first_prev"):
        rmd.sample_block_tokens_processed(x, torch.zeros(3, dtype=torch.int64), torch.zeros(40, 8), torch.zeros(40, 8))


def test_rules_arguments_are_checked():
    cuda = torch.device("cuda", 0)
    i64 = dict(dtype=torch.int64)

    def r(**kw):
        names = ("history", "lengths", "prompt_lengths", "repetition_penalty", "frequency_penalty", "presence_penalty",
                 "logit_bias", "token_mask")
        return rmd._logit_rules(2, 3, 40, cuda, *(kw.get(n) for n in names))
    r()
    for kw, err in ((dict(history=torch.zeros(3, 4, **i64)), ValueError), (dict(history=torch.zeros(2, 4)), ValueError),
                    (dict(lengths=torch.zeros(2, **i64)), ValueError),
                    (dict(history=torch.zeros(2, 4, **i64), lengths=torch.zeros(3, **i64)), ValueError),
                    (dict(history=torch.zeros(2, 4, **i64), lengths=torch.zeros(2)), TypeError),
                    (dict(repetition_penalty=torch.ones(1)), ValueError),
                    (dict(presence_penalty=torch.ones(2, **i64)), TypeError),
                    (dict(logit_bias=torch.zeros(39)), ValueError), (dict(logit_bias=torch.zeros(3, 40)), ValueError),
                    (dict(logit_bias=torch.zeros(40, dtype=torch.float64)), TypeError),
                    (dict(token_mask=torch.zeros(2, 2, **i64)), TypeError),
                    (dict(token_mask=torch.zeros(2, 3, dtype=torch.int32)), ValueError),
                    (dict(token_mask=torch.zeros(2, 2, 2, dtype=torch.int32)), ValueError),
                    (dict(token_mask=torch.zeros(2, 2, dtype=torch.int32)), ValueError)):   # on the host
        with pytest.raises(err):
            r(**kw)
