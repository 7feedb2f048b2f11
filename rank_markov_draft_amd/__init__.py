"""DSpark low-rank Markov head on MI355X (gfx950).

Python binding of libdspark_markov.so with the names of the pages'
VanillaMarkov methods (third-party markov_head.py page):

* ``apply_block_logits(base_logits, token_ids, w1, w2)`` -- teacher-forced
  bias of every block position by its given predecessor;
* ``sample_block_tokens(base_logits, first_prev_token_ids, w1, w2,
  temperature=0.0, ...)`` -- left-to-right sampling, each position biased by
  the token drawn at the previous one.

``apply_block_logits_backward`` gives the gradients of W1 and W2 for a
gradient of the teacher-forced corrected logits (training).
``apply_block_logits_lm_head`` fuses the drafter's FP32 vocabulary head
(the base logits) with the teacher-forced bias.

The gated head (the pages' GatedMarkovHead) has the same two operations,
``apply_block_logits_gated`` and ``sample_block_tokens_gated``, which also
take the backbone hidden states and the gate_proj weight and bias.

For serving, ``lm_head_logits_int8`` computes base logits with the vocabulary
head held in 8-bit integers (``quantize_rows`` makes them), and
``process_block_logits`` applies a request's penalties for repeated tokens,
biases and grammar masks to logits, ``sample_block_tokens_processed`` within
the left-to-right draft; ``process_block_logits_backward`` is the rules'
gradient.

Tensors must live on the current HIP device.  ``w1`` is the Embedding
weight [V, r]; ``w2`` is the Linear(r, V) weight [V, r].  This module only
marshals arguments (dtype tags, pointers, sizes, the current stream) and
allocates outputs and workspace with torch: every step of the computation
runs in the library's kernels.  There is no fallback path: if the library
is missing, the first call raises.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib

__all__ = ["apply_block_logits", "sample_block_tokens", "apply_block_logits_gated",
           "sample_block_tokens_gated", "apply_block_logits_backward", "apply_block_logits_lm_head",
           "quantize_rows", "lm_head_logits_int8", "process_block_logits", "process_block_logits_backward",
           "sample_block_tokens_processed", "Workspace",
           "read_device_error", "workspace_bytes"]


def _dtype_tag(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return _lib.DSPARK_F32
    if t.dtype == torch.bfloat16:
        return _lib.DSPARK_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; the head takes float32 or bfloat16")


def _stream_handle(device: torch.device) -> int:
    # the hipStream_t of torch's current stream, without the Stream object
    # that torch.cuda.current_stream would build (2 us of a small call's 14)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device.index is None else device.index)


def _call(device: torch.device, fn, *args) -> int:
    """fn(*args, stream) with ``device`` the current one."""
    if torch.cuda.current_device() == device.index:
        return fn(*args, _stream_handle(device))
    with torch.cuda.device(device):
        return fn(*args, _stream_handle(device))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def workspace_bytes(B: int, M: int, V: int, r: int, sample: bool, hidden: int | None = None) -> int:
    """Workspace bytes of a call; ``hidden`` (the hidden size d, or 0 for the
    gated calls' vanilla fallback) sizes it for the gated calls."""
    if hidden is None:
        return int(_lib.load().dspark_markov_workspace_bytes(B, M, V, r, 1 if sample else 0))
    return int(_lib.load().dspark_markov_gated_workspace_bytes(B, M, V, r, hidden, 1 if sample else 0))


class Workspace:
    """Device workspace for a family of calls of at most the given sizes
    (``hidden``: the hidden size of gated calls; ``backward``: sized for the
    backward as well; ``int8_hidden``: the hidden size of 8-bit head calls;
    ``processed``: sized for sampling under logit rules as well).

    Zero-filled once at creation; the library leaves it ready for the next
    call.  Calls sharing one workspace must be ordered on one stream."""

    def __init__(self, B: int, M: int, V: int, r: int, sample: bool, device=None,
                 hidden: int | None = None, backward: bool = False, int8_hidden: int | None = None,
                 processed: bool = False):
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"the head runs on a GPU; the workspace would be on {device}")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.nbytes = max(workspace_bytes(B, M, V, r, sample, hidden), 256)
        if backward:
            self.nbytes = max(self.nbytes, int(_lib.load().dspark_markov_backward_workspace_bytes(B, M, V, r)))
        if int8_hidden is not None:
            self.nbytes = max(self.nbytes, int(_lib.load().dspark_markov_lm_head_int8_workspace_bytes(B, M, int8_hidden)))
        if processed:
            self.nbytes = max(self.nbytes, int(_lib.load().dspark_markov_processed_workspace_bytes(B, M, V, r)))
        self.device = device
        self.buffer = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        _lib.check(_call(device, _lib.load().dspark_markov_workspace_init, _ptr(self.buffer), self.nbytes),
                   "workspace_init")

    @property
    def ptr(self):
        return _ptr(self.buffer)

    def set_chain_test_hook(self, on: bool):
        """Tests of the failure path: with the hook on, the persistent chain's
        device-wide waits give up at once, so the call returns -1 tokens and
        records a failure without a stall (control word at byte 128)."""
        self.buffer[128:132].view(torch.int32).fill_(1 if on else 0)


def read_device_error(ws: Workspace) -> int:
    """Rows with out-of-range predecessor ids since the last read (synchronises).
    Raises DeviceError when a persistent sampling launch on ``ws`` failed since
    the last read (its tokens were -1); the record is cleared either way."""
    n = ctypes.c_int64(0)
    with torch.cuda.device(ws.device):
        _lib.check(_lib.load().dspark_markov_read_device_error(
            ws.ptr, _stream_handle(ws.device), ctypes.byref(n)), "read_device_error")
    return int(n.value)


def _check_weights(w1: torch.Tensor, w2: torch.Tensor):
    if w1.dim() != 2 or w2.dim() != 2 or w1.shape != w2.shape:
        raise ValueError(f"w1 and w2 must both be [V, r], got {tuple(w1.shape)} and {tuple(w2.shape)}")
    if w1.dtype != w2.dtype:
        raise TypeError("w1 and w2 must share a dtype")


def apply_block_logits(base_logits: torch.Tensor, token_ids: torch.Tensor, w1: torch.Tensor,
                       w2: torch.Tensor, *, out: torch.Tensor | None = None,
                       workspace: Workspace | None = None) -> torch.Tensor:
    """Teacher-forced corrected logits base[..., M, V] + bias(token_ids[..., M]).

    ``out`` may be ``base_logits`` itself (in place).  An empty input returns
    ``base_logits`` (or ``out`` untouched), as the pages' method does."""
    _check_weights(w1, w2)
    if base_logits.dim() < 2:
        raise ValueError("base_logits must be [..., M, V]")
    V = base_logits.shape[-1]
    M = base_logits.shape[-2]
    B = 1
    for d in base_logits.shape[:-2]:
        B *= int(d)
    if tuple(token_ids.shape) != tuple(base_logits.shape[:-1]):
        raise ValueError(f"token_ids {tuple(token_ids.shape)} must be base_logits.shape[:-1]")
    if w1.shape[0] != V:
        raise ValueError(f"weights have vocabulary {w1.shape[0]}, logits {V}")
    _check_device(base_logits.device, workspace, token_ids=token_ids, w1=w1, w2=w2, out=out)
    if base_logits.numel() == 0:
        return base_logits if out is None else out
    base_c = base_logits.contiguous()
    ids = token_ids.to(torch.int64).contiguous()
    w1c, w2c = w1.contiguous(), w2.contiguous()
    if out is None:
        out = torch.empty_like(base_c)
    elif out.shape != base_logits.shape or out.dtype != base_logits.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor shaped and typed like base_logits")
    r = w1.shape[1]
    if workspace is None:
        workspace = Workspace(B, M, V, r, sample=False, device=base_c.device)
    st = _lib.load().dspark_markov_apply_block(
        _ptr(base_c), _dtype_tag(base_c), _ptr(ids), _ptr(w1c), _ptr(w2c), _dtype_tag(w1c),
        B, M, V, r, _ptr(out), workspace.ptr, workspace.nbytes, _stream_handle(base_c.device))
    _lib.check(st, "apply_block_logits")
    return out


def sample_block_tokens(base_logits: torch.Tensor, first_prev_token_ids: torch.Tensor,
                        w1: torch.Tensor, w2: torch.Tensor, temperature: float | None = 0.0, *,
                        seed: int = 0, position_offset: int = 0, batch_offset: int = 0,
                        return_logits: bool = True, tokens_out: torch.Tensor | None = None,
                        logits_out: torch.Tensor | None = None,
                        workspace: Workspace | None = None, check: bool = False):
    """Left-to-right block sampling over base_logits [B, M, V].

    Returns ``(sampled_tokens [B, M] int64, corrected_logits [B, M, V] or None)``.
    ``temperature`` None or below 1e-5 is greedy argmax; otherwise Gumbel-max
    with Philox4x32-10 noise keyed by ``seed``.

    Greedy bf16 calls of up to 64 rows run as one persistent launch.  If its
    workgroups cannot all run (CUs held by other work), it gives up after 1 s
    and every token is -1; later persistent calls on the same workspace also
    return -1 tokens until ``read_device_error`` (which raises) clears the
    record.  ``check=True`` synchronises after the call and raises at once."""
    _check_weights(w1, w2)
    if base_logits.dim() != 3:
        raise ValueError("base_logits must be [B, M, V]")
    B, M, V = base_logits.shape
    if tuple(first_prev_token_ids.shape) != (B,):
        raise ValueError("first_prev_token_ids must be [B]")
    if w1.shape[0] != V:
        raise ValueError(f"weights have vocabulary {w1.shape[0]}, logits {V}")
    T = 0.0 if temperature is None else float(temperature)
    dev = base_logits.device
    _check_device(dev, workspace, first_prev_token_ids=first_prev_token_ids, w1=w1, w2=w2,
                  tokens_out=tokens_out, logits_out=logits_out if return_logits else None)
    if tokens_out is not None and (tuple(tokens_out.shape) != (B, M) or tokens_out.dtype != torch.int64
                                   or not tokens_out.is_contiguous()):
        raise ValueError(f"tokens_out must be a contiguous int64 tensor of shape {(B, M)}")
    if return_logits and logits_out is not None and (
            logits_out.shape != base_logits.shape or logits_out.dtype != base_logits.dtype
            or not logits_out.is_contiguous()):
        raise ValueError("logits_out must be a contiguous tensor shaped and typed like base_logits")
    if tokens_out is None:
        tokens_out = torch.empty((B, M), dtype=torch.int64, device=dev)
    if M == 0:
        return tokens_out, (base_logits if return_logits else None)
    base_c = base_logits.contiguous()
    first = first_prev_token_ids.to(torch.int64).contiguous()
    w1c, w2c = w1.contiguous(), w2.contiguous()
    corrected = None
    if return_logits:
        corrected = torch.empty_like(base_c) if logits_out is None else logits_out
    r = w1.shape[1]
    if workspace is None:
        workspace = Workspace(B, M, V, r, sample=True, device=dev)
    st = _lib.load().dspark_markov_sample_block(
        _ptr(base_c), _dtype_tag(base_c), _ptr(first), _ptr(w1c), _ptr(w2c), _dtype_tag(w1c),
        B, M, V, r, T, int(seed) & (2**64 - 1), int(position_offset), int(batch_offset),
        _ptr(tokens_out), _ptr(corrected), workspace.ptr, workspace.nbytes, _stream_handle(dev))
    _lib.check(st, "sample_block_tokens")
    if check:
        read_device_error(workspace)
    return tokens_out, corrected


def apply_block_logits_lm_head(hidden_states: torch.Tensor, lm_head_weight: torch.Tensor,
                               token_ids: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, *,
                               out: torch.Tensor | None = None,
                               workspace: Workspace | None = None) -> torch.Tensor:
    """The drafter's vocabulary head fused with the teacher-forced bias:
    hidden_states [..., M, d] and the head's Linear weight [V, d] give FP32
    base logits U (DeepseekV41DSparkModel.compute_logits), and the result is
    U + bias(token_ids[..., M]) as apply_block_logits would return it, in
    float32 [..., M, V], without U being materialised."""
    _check_weights(w1, w2)
    if hidden_states.dim() < 2:
        raise ValueError("hidden_states must be [..., M, d]")
    d = hidden_states.shape[-1]
    M = hidden_states.shape[-2]
    B = 1
    for x in hidden_states.shape[:-2]:
        B *= int(x)
    V, r = w1.shape
    if lm_head_weight.dim() != 2 or tuple(lm_head_weight.shape) != (V, d):
        raise ValueError(f"lm_head_weight must be [V, d] = {(V, d)}, got {tuple(lm_head_weight.shape)}")
    if tuple(token_ids.shape) != tuple(hidden_states.shape[:-1]):
        raise ValueError(f"token_ids {tuple(token_ids.shape)} must be hidden_states.shape[:-1]")
    dev = hidden_states.device
    _check_device(dev, workspace, lm_head_weight=lm_head_weight, token_ids=token_ids, w1=w1, w2=w2, out=out)
    shape = tuple(hidden_states.shape[:-1]) + (V,)
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=dev)
    elif tuple(out.shape) != shape or out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous float32 tensor of shape {shape}")
    if out.numel() == 0:
        return out
    h = hidden_states.contiguous()
    lm = lm_head_weight.contiguous()
    ids = token_ids.to(torch.int64).contiguous()
    w1c, w2c = w1.contiguous(), w2.contiguous()
    if workspace is None:
        workspace = Workspace(B, M, V, r, sample=False, device=dev)
    st = _lib.load().dspark_markov_apply_block_lm_head(
        _ptr(h), _dtype_tag(h), d, _ptr(lm), _dtype_tag(lm), _ptr(ids), _ptr(w1c), _ptr(w2c), _dtype_tag(w1c),
        B, M, V, r, _ptr(out), workspace.ptr, workspace.nbytes, _stream_handle(dev))
    _lib.check(st, "apply_block_logits_lm_head")
    return out


def _check_device(dev: torch.device, workspace: "Workspace | None" = None, **tensors):
    """Every tensor the kernels read or write must live on the GPU that holds
    the logits: a host or foreign-device pointer would reach the kernels."""
    if dev.type != "cuda":
        raise ValueError(f"the head runs on a GPU; the logits are on {dev}")
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the logits on {dev}")
    if workspace is not None and workspace.buffer.device != dev:
        raise ValueError(f"the workspace is on {workspace.buffer.device}, the logits on {dev}")


def _check_gate(hidden_states, gate_weight, gate_bias, lead, d_expected_rows, r, wdtype):
    if hidden_states is None:
        return 0
    if tuple(hidden_states.shape[:-1]) != tuple(lead):
        raise ValueError(f"hidden_states {tuple(hidden_states.shape)} must be {tuple(lead)} + (d,)")
    d = hidden_states.shape[-1]
    if gate_weight is None or gate_bias is None:
        raise ValueError("the gated head needs gate_weight [r, d + r] and gate_bias [r]")
    if tuple(gate_weight.shape) != (r, d + r) or tuple(gate_bias.shape) != (r,):
        raise ValueError(f"gate_weight must be [{r}, {d + r}] and gate_bias [{r}]")
    if gate_weight.dtype != wdtype or gate_bias.dtype != wdtype:
        raise TypeError("gate_weight and gate_bias must have the dtype of w1 and w2")
    return d


def apply_block_logits_gated(base_logits: torch.Tensor, token_ids: torch.Tensor, w1: torch.Tensor,
                             w2: torch.Tensor, gate_weight: torch.Tensor | None,
                             gate_bias: torch.Tensor | None, hidden_states: torch.Tensor | None, *,
                             out: torch.Tensor | None = None, return_latent: bool = False,
                             workspace: Workspace | None = None):
    """Teacher-forced corrected logits of the gated head (GatedMarkovHead):
    base[..., M, V] + W2 (sigmoid(gate_proj([h; W1[x]])) * W1[x]).

    ``hidden_states`` [..., M, d]; None is the pages' vanilla fallback.
    Returns the corrected logits, and with ``return_latent`` also the latent
    rows [..., M, r] the projection consumed."""
    _check_weights(w1, w2)
    if base_logits.dim() < 2:
        raise ValueError("base_logits must be [..., M, V]")
    V, M = base_logits.shape[-1], base_logits.shape[-2]
    B = 1
    for s_ in base_logits.shape[:-2]:
        B *= int(s_)
    if tuple(token_ids.shape) != tuple(base_logits.shape[:-1]):
        raise ValueError(f"token_ids {tuple(token_ids.shape)} must be base_logits.shape[:-1]")
    if w1.shape[0] != V:
        raise ValueError(f"weights have vocabulary {w1.shape[0]}, logits {V}")
    r = w1.shape[1]
    d = _check_gate(hidden_states, gate_weight, gate_bias, base_logits.shape[:-1], None, r, w1.dtype)
    dev = base_logits.device
    gated = hidden_states is not None
    _check_device(dev, workspace, token_ids=token_ids, w1=w1, w2=w2, hidden_states=hidden_states, out=out,
                  gate_weight=gate_weight if gated else None, gate_bias=gate_bias if gated else None)
    latent = torch.empty(tuple(base_logits.shape[:-1]) + (r,), dtype=w1.dtype, device=dev) if return_latent else None
    if base_logits.numel() == 0:
        res = base_logits if out is None else out
        return (res, latent) if return_latent else res
    base_c = base_logits.contiguous()
    ids = token_ids.to(torch.int64).contiguous()
    w1c, w2c = w1.contiguous(), w2.contiguous()
    hc = hidden_states.contiguous() if hidden_states is not None else None
    gwc = gate_weight.contiguous() if hc is not None else None
    gbc = gate_bias.contiguous() if hc is not None else None
    if out is None:
        out = torch.empty_like(base_c)
    elif out.shape != base_logits.shape or out.dtype != base_logits.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor shaped and typed like base_logits")
    if workspace is None:
        workspace = Workspace(B, M, V, r, sample=False, device=dev, hidden=d)
    st = _lib.load().dspark_markov_apply_block_gated(
        _ptr(base_c), _dtype_tag(base_c), _ptr(ids), _ptr(hc), _dtype_tag(hc) if hc is not None else 0, d,
        _ptr(w1c), _ptr(w2c), _ptr(gwc), _ptr(gbc), _dtype_tag(w1c), B, M, V, r, _ptr(out), _ptr(latent),
        workspace.ptr, workspace.nbytes, _stream_handle(dev))
    _lib.check(st, "apply_block_logits_gated")
    return (out, latent) if return_latent else out


def sample_block_tokens_gated(base_logits: torch.Tensor, first_prev_token_ids: torch.Tensor,
                              w1: torch.Tensor, w2: torch.Tensor, gate_weight: torch.Tensor | None,
                              gate_bias: torch.Tensor | None, hidden_states: torch.Tensor | None,
                              temperature: float | None = 0.0, *, seed: int = 0, position_offset: int = 0,
                              batch_offset: int = 0, return_logits: bool = True,
                              return_latent: bool = False, workspace: Workspace | None = None):
    """Left-to-right sampling with the gated head; step k gates with
    hidden_states[:, k, :] ([B, M, d]; None: vanilla fallback) and the token
    drawn at k - 1.  Returns (tokens [B, M], corrected [B, M, V] or None) and,
    with ``return_latent``, the latent rows [B, M, r] as a third item."""
    _check_weights(w1, w2)
    if base_logits.dim() != 3:
        raise ValueError("base_logits must be [B, M, V]")
    B, M, V = base_logits.shape
    if tuple(first_prev_token_ids.shape) != (B,):
        raise ValueError("first_prev_token_ids must be [B]")
    if w1.shape[0] != V:
        raise ValueError(f"weights have vocabulary {w1.shape[0]}, logits {V}")
    r = w1.shape[1]
    d = _check_gate(hidden_states, gate_weight, gate_bias, (B, M), None, r, w1.dtype)
    T = 0.0 if temperature is None else float(temperature)
    dev = base_logits.device
    gated = hidden_states is not None
    _check_device(dev, workspace, first_prev_token_ids=first_prev_token_ids, w1=w1, w2=w2,
                  hidden_states=hidden_states, gate_weight=gate_weight if gated else None,
                  gate_bias=gate_bias if gated else None)
    tokens = torch.empty((B, M), dtype=torch.int64, device=dev)
    latent = torch.empty((B, M, r), dtype=w1.dtype, device=dev) if return_latent else None
    if M == 0 or B == 0:
        res = (tokens, base_logits if return_logits else None)
        return res + (latent,) if return_latent else res
    base_c = base_logits.contiguous()
    first = first_prev_token_ids.to(torch.int64).contiguous()
    w1c, w2c = w1.contiguous(), w2.contiguous()
    hc = hidden_states.contiguous() if hidden_states is not None else None
    gwc = gate_weight.contiguous() if hc is not None else None
    gbc = gate_bias.contiguous() if hc is not None else None
    corrected = torch.empty_like(base_c) if return_logits else None
    if workspace is None:
        workspace = Workspace(B, M, V, r, sample=True, device=dev, hidden=d)
    st = _lib.load().dspark_markov_sample_block_gated(
        _ptr(base_c), _dtype_tag(base_c), _ptr(first), _ptr(hc), _dtype_tag(hc) if hc is not None else 0, d,
        _ptr(w1c), _ptr(w2c), _ptr(gwc), _ptr(gbc), _dtype_tag(w1c), B, M, V, r, T, int(seed) & (2**64 - 1),
        int(position_offset), int(batch_offset), _ptr(tokens), _ptr(corrected), _ptr(latent),
        workspace.ptr, workspace.nbytes, _stream_handle(dev))
    _lib.check(st, "sample_block_tokens_gated")
    return (tokens, corrected, latent) if return_latent else (tokens, corrected)


def apply_block_logits_backward(grad_corrected: torch.Tensor, token_ids: torch.Tensor, w1: torch.Tensor,
                                w2: torch.Tensor, *, workspace: Workspace | None = None):
    """Gradients (grad_w1 [V, r], grad_w2 [V, r]) of the teacher-forced apply
    for the gradient of the corrected logits grad_corrected [..., M, V]; the
    base logits' gradient is grad_corrected itself."""
    _check_weights(w1, w2)
    if grad_corrected.dim() < 2:
        raise ValueError("grad_corrected must be [..., M, V]")
    V, M = grad_corrected.shape[-1], grad_corrected.shape[-2]
    B = 1
    for s_ in grad_corrected.shape[:-2]:
        B *= int(s_)
    if tuple(token_ids.shape) != tuple(grad_corrected.shape[:-1]):
        raise ValueError(f"token_ids {tuple(token_ids.shape)} must be grad_corrected.shape[:-1]")
    if w1.shape[0] != V:
        raise ValueError(f"weights have vocabulary {w1.shape[0]}, logits {V}")
    r = w1.shape[1]
    dev = grad_corrected.device
    _check_device(dev, workspace, token_ids=token_ids, w1=w1, w2=w2)
    g = grad_corrected.contiguous()
    ids = token_ids.to(torch.int64).contiguous()
    w1c, w2c = w1.contiguous(), w2.contiguous()
    gw1 = torch.empty_like(w1c)
    gw2 = torch.empty_like(w2c)
    if workspace is None:
        workspace = Workspace(B, M, V, r, sample=False, device=dev, backward=True)
    st = _lib.load().dspark_markov_apply_block_backward(
        _ptr(g), _dtype_tag(g), _ptr(ids), _ptr(w1c), _ptr(w2c), _dtype_tag(w1c), B, M, V, r, _ptr(gw1), _ptr(gw2),
        workspace.ptr, workspace.nbytes, _stream_handle(dev))
    _lib.check(st, "apply_block_logits_backward")
    return gw1, gw2


def quantize_rows(x: torch.Tensor, *, out: torch.Tensor | None = None, scale_out: torch.Tensor | None = None):
    """Rows of 8-bit integers with one fp32 scale each: x [..., d] gives
    ``(q [..., d] int8, scale [...])`` with scale = max|x| / 127 and
    q = clamp(rint(x / scale), -127, 127).  A row of zeros has scale 0; a row
    with an infinity or NaN has it as its scale (and zeros), so that what is
    computed from the row shows it."""
    if x.dim() < 1:
        raise ValueError("x must be [..., d]")
    _check_device(x.device, None, out=out, scale_out=scale_out)
    tag = _dtype_tag(x)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    elif out.shape != x.shape or out.dtype != torch.int8 or not out.is_contiguous():
        raise ValueError("out must be a contiguous int8 tensor shaped like x")
    if scale_out is None:
        scale_out = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    elif scale_out.shape != x.shape[:-1] or scale_out.dtype != torch.float32 or not scale_out.is_contiguous():
        raise ValueError(f"scale_out must be a contiguous float32 tensor of shape {tuple(x.shape[:-1])}")
    xc = x.contiguous()
    st = _call(x.device, _lib.load().dspark_markov_quantize_rows, _ptr(xc), tag, scale_out.numel(), x.shape[-1],
               _ptr(out), _ptr(scale_out))
    _lib.check(st, "quantize_rows")
    return out, scale_out


def lm_head_logits_int8(hidden_states: torch.Tensor, head_q: torch.Tensor, head_scale: torch.Tensor, *,
                        out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                        workspace: Workspace | None = None) -> torch.Tensor:
    """Base logits [..., V] of hidden_states [..., d] through a vocabulary head
    held in 8-bit integers: head_q [V, d] and head_scale [V] as quantize_rows
    gives them for the head's Linear weight.  The hidden states are quantised
    row by row in the call (one scale for each token), the products summed
    exactly in 32-bit integers.  ``out_dtype``: float32 (default) or bfloat16."""
    if hidden_states.dim() < 1:
        raise ValueError("hidden_states must be [..., d]")
    d = hidden_states.shape[-1]
    if head_q.dim() != 2 or head_q.shape[1] != d or head_q.dtype != torch.int8:
        raise ValueError(f"head_q must be int8 [V, {d}], got {head_q.dtype} {tuple(head_q.shape)}")
    V = head_q.shape[0]
    if tuple(head_scale.shape) != (V,) or head_scale.dtype != torch.float32:
        raise ValueError(f"head_scale must be float32 [{V}], got {head_scale.dtype} {tuple(head_scale.shape)}")
    dev = hidden_states.device
    _check_device(dev, workspace, head_q=head_q, head_scale=head_scale, out=out)
    tag = _dtype_tag(hidden_states)
    shape = tuple(hidden_states.shape[:-1]) + (V,)
    if out_dtype is None:
        out_dtype = torch.float32 if out is None else out.dtype
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=dev)
    elif tuple(out.shape) != shape or out.dtype != out_dtype or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {out_dtype} tensor of shape {shape}")
    out_tag = _dtype_tag(out)
    if out.numel() == 0:
        return out
    rows = out.numel() // V
    h, hq, hs = hidden_states.contiguous(), head_q.contiguous(), head_scale.contiguous()
    if workspace is None:
        nbytes = int(_lib.load().dspark_markov_lm_head_int8_workspace_bytes(rows, 1, d))
        buffer = torch.empty(nbytes, dtype=torch.uint8, device=dev)  # needs no zero fill
    else:
        nbytes, buffer = workspace.nbytes, workspace.buffer
    st = _call(dev, _lib.load().dspark_markov_lm_head_int8, _ptr(h), tag, d, _ptr(hq), _ptr(hs), rows, 1, V, _ptr(out),
               out_tag, _ptr(buffer), nbytes)
    _lib.check(st, "lm_head_logits_int8")
    return out


def _logit_rules(B, M, V, dev, history, lengths, prompt_lengths, repetition_penalty, frequency_penalty, presence_penalty,
                 logit_bias, token_mask):
    """The rules as dspark_logit_rules_t, and the tensors made for it that must live until the call."""
    r, keep, given = _lib.LogitRules(), [], {}

    def per_request(t, name, dtype):
        if t is None:
            return None
        if t.shape != (B,):
            raise ValueError(f"{name} must be [{B}], got {tuple(t.shape)}")
        if t.is_floating_point() != dtype.is_floating_point:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        given[name] = t
        if t.dtype != dtype or not t.is_contiguous():
            t = t.to(dtype).contiguous()
            keep.append(t)
        return t.data_ptr()

    if history is not None:
        if history.dim() != 2 or history.shape[0] != B or history.is_floating_point():
            raise ValueError(f"history must be integer ids [{B}, L], got {history.dtype} {tuple(history.shape)}")
        given["history"] = history
        L = history.shape[1]
        if history.dtype != torch.int64 or L > 1 and history.stride(1) != 1 or B > 1 and history.stride(0) < L:
            history = history.to(torch.int64).contiguous()
            keep.append(history)
        r.history, r.history_len, r.history_stride = history.data_ptr(), L, history.stride(0) if B > 1 else L
        r.lengths = per_request(lengths, "lengths", torch.int64)
        r.prompt_lengths = per_request(prompt_lengths, "prompt_lengths", torch.int64)
    elif lengths is not None or prompt_lengths is not None:
        raise ValueError("lengths and prompt_lengths need a history")
    r.repetition_penalty = per_request(repetition_penalty, "repetition_penalty", torch.float32)
    r.frequency_penalty = per_request(frequency_penalty, "frequency_penalty", torch.float32)
    r.presence_penalty = per_request(presence_penalty, "presence_penalty", torch.float32)
    if logit_bias is not None:
        if tuple(logit_bias.shape) not in ((V,), (1, V), (B, V)):
            raise ValueError(f"logit_bias must be [{V}] or [{B}, {V}], got {tuple(logit_bias.shape)}")
        r.bias_dtype = _dtype_tag(logit_bias)
        given["logit_bias"] = logit_bias
        if not logit_bias.is_contiguous():
            logit_bias = logit_bias.contiguous()
            keep.append(logit_bias)
        r.logit_bias = logit_bias.data_ptr()
        r.bias_stride = V if logit_bias.dim() == 2 and logit_bias.shape[0] > 1 else 0
    if token_mask is not None:
        W = (V + 31) // 32
        if token_mask.dtype != torch.int32:
            raise TypeError(f"token_mask must be int32 words of 32 tokens, got {token_mask.dtype}")
        mask = token_mask[:, None] if token_mask.dim() == 2 else token_mask
        if mask.dim() != 3 or mask.shape[0] not in (1, B) or mask.shape[1] not in (1, M) or mask.shape[2] != W:
            raise ValueError(f"token_mask must be [{B}, {W}] or [{B}, {M}, {W}] (or 1 in place of either size), "
                             f"got {tuple(token_mask.shape)}")
        given["token_mask"] = token_mask
        if W > 1 and mask.stride(2) != 1:
            mask = mask.contiguous()
            keep.append(mask)
        r.token_mask = mask.data_ptr()
        r.mask_stride_b = mask.stride(0) if mask.shape[0] > 1 else 0
        r.mask_stride_m = mask.stride(1) if mask.shape[1] > 1 else 0
    for name, t in given.items():
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the logits on {dev}")
    return r, keep


def _block(logits, token_ids, what):
    if logits.dim() != 3:
        raise ValueError(f"{what} must be [B, M, V]")
    if token_ids is not None and (tuple(token_ids.shape) != tuple(logits.shape[:2]) or token_ids.is_floating_point()):
        raise ValueError(f"token_ids must be integer ids of shape {tuple(logits.shape[:2])}")
    return logits.shape


def process_block_logits(logits: torch.Tensor, *, token_ids: torch.Tensor | None = None,
                         history: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
                         prompt_lengths: torch.Tensor | None = None, repetition_penalty: torch.Tensor | None = None,
                         frequency_penalty: torch.Tensor | None = None, presence_penalty: torch.Tensor | None = None,
                         logit_bias: torch.Tensor | None = None, token_mask: torch.Tensor | None = None,
                         out: torch.Tensor | None = None) -> torch.Tensor:
    """Penalties for repeated tokens, biases and grammar masks on logits
    [B, M, V] (M = 1: a single token each).  For a token that stands in the
    request's counted tokens x becomes x / repetition_penalty (x > 0) or
    x * repetition_penalty; for one that stands c times among its outputs
    frequency_penalty * c + presence_penalty is taken off; then the bias is
    added; a masked token is -inf.  fp32 arithmetic, one rounding.

    ``history`` [B, L]: each request's tokens, prompt first; ``lengths`` [B]
    how many count (default: all; what lies behind is not read; ids outside
    the vocabulary are ignored), ``prompt_lengths`` [B] how many of them are
    the prompt's (default: none), which only the repetition penalty sees.
    ``token_ids`` [B, M]: the predecessors of apply_block_logits; at position k
    the tokens token_ids[:, 1 .. k] count as outputs too (the first is the
    history's last).  The penalties are [B]; ``logit_bias`` [V] or [B, V];
    ``token_mask`` int32 words of 32 tokens, [B, W] or [B, M, W] (either size
    may be 1), bit set: allowed.  Rules not given are off.  ``out`` may be
    ``logits`` itself (in place)."""
    B, M, V = _block(logits, token_ids, "logits")
    dev = logits.device
    _check_device(dev, None, token_ids=token_ids, out=out)
    tag = _dtype_tag(logits)
    rules, keep = _logit_rules(B, M, V, dev, history, lengths, prompt_lengths, repetition_penalty, frequency_penalty,
                               presence_penalty, logit_bias, token_mask)
    x = logits.contiguous()
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != logits.shape or out.dtype != logits.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor shaped and typed like logits")
    ids = None if token_ids is None else token_ids.to(torch.int64).contiguous()
    st = _call(dev, _lib.load().dspark_markov_process_block, _ptr(x), tag, _ptr(ids), rules, B, M, V, _ptr(out))
    _lib.check(st, "process_block_logits")
    return out


def process_block_logits_backward(grad_processed: torch.Tensor, logits: torch.Tensor, *,
                                  token_ids: torch.Tensor | None = None, history: torch.Tensor | None = None,
                                  lengths: torch.Tensor | None = None, prompt_lengths: torch.Tensor | None = None,
                                  repetition_penalty: torch.Tensor | None = None,
                                  token_mask: torch.Tensor | None = None,
                                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of the logits [B, M, V] for the gradient of what
    process_block_logits made of them: 0 where masked, the repetition
    penalty's slope where the token was seen (1 / penalty for a logit above
    zero, else the penalty), else the gradient itself.  ``logits`` and the
    rules as in the forward call (frequency and presence penalties and biases
    only shift, so they are not asked for); ``out`` may be
    ``grad_processed`` itself."""
    B, M, V = _block(logits, token_ids, "logits")
    if grad_processed.shape != logits.shape or grad_processed.dtype != logits.dtype:
        raise ValueError("grad_processed must be shaped and typed like logits")
    dev = logits.device
    _check_device(dev, None, grad_processed=grad_processed, token_ids=token_ids, out=out)
    tag = _dtype_tag(logits)
    rules, keep = _logit_rules(B, M, V, dev, history, lengths, prompt_lengths, repetition_penalty, None, None, None,
                               token_mask)
    g, x = grad_processed.contiguous(), logits.contiguous()
    if out is None:
        out = torch.empty_like(g)
    elif out.shape != logits.shape or out.dtype != logits.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor shaped and typed like logits")
    ids = None if token_ids is None else token_ids.to(torch.int64).contiguous()
    st = _call(dev, _lib.load().dspark_markov_process_block_backward, _ptr(g), _ptr(x), tag, _ptr(ids), rules, B, M, V,
               _ptr(out))
    _lib.check(st, "process_block_logits_backward")
    return out


def sample_block_tokens_processed(base_logits: torch.Tensor, first_prev_token_ids: torch.Tensor, w1: torch.Tensor,
                                  w2: torch.Tensor, temperature: float | None = 0.0, *,
                                  history: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
                                  prompt_lengths: torch.Tensor | None = None,
                                  repetition_penalty: torch.Tensor | None = None,
                                  frequency_penalty: torch.Tensor | None = None,
                                  presence_penalty: torch.Tensor | None = None,
                                  logit_bias: torch.Tensor | None = None, token_mask: torch.Tensor | None = None,
                                  seed: int = 0, position_offset: int = 0, batch_offset: int = 0,
                                  tokens_out: torch.Tensor | None = None, logits_out: torch.Tensor | None = None,
                                  workspace: Workspace | None = None, check: bool = False):
    """sample_block_tokens under the rules of process_block_logits: position k
    draws from the processed corrected logits, and the tokens drawn before it
    count as outputs beside ``history`` (which ends with
    first_prev_token_ids).  Returns ``(tokens [B, M], processed [B, M, V])``.
    A row left with nothing above -inf gets token -1 (the position after it
    then has no bias).  M = 1 with ``position_offset`` is the single-token
    form, for masks that depend on the tokens drawn.

    Greedy bf16 drafts of up to 64 rows without per-request biases run as one
    persistent launch that needs every compute unit within a second, as
    sample_block_tokens' do: if another stream holds some for longer, every
    token is -1 and read_device_error(workspace) raises.  ``check=True``
    synchronises after the call and raises at once."""
    _check_weights(w1, w2)
    B, M, V = _block(base_logits, None, "base_logits")
    if tuple(first_prev_token_ids.shape) != (B,):
        raise ValueError("first_prev_token_ids must be [B]")
    if w1.shape[0] != V:
        raise ValueError(f"weights have vocabulary {w1.shape[0]}, logits {V}")
    T = 0.0 if temperature is None else float(temperature)
    dev = base_logits.device
    _check_device(dev, workspace, first_prev_token_ids=first_prev_token_ids, w1=w1, w2=w2, tokens_out=tokens_out,
                  logits_out=logits_out)
    tag, wtag = _dtype_tag(base_logits), _dtype_tag(w1)
    rules, keep = _logit_rules(B, M, V, dev, history, lengths, prompt_lengths, repetition_penalty, frequency_penalty,
                               presence_penalty, logit_bias, token_mask)
    if tokens_out is None:
        tokens_out = torch.empty((B, M), dtype=torch.int64, device=dev)
    elif tuple(tokens_out.shape) != (B, M) or tokens_out.dtype != torch.int64 or not tokens_out.is_contiguous():
        raise ValueError(f"tokens_out must be a contiguous int64 tensor of shape {(B, M)}")
    if logits_out is None:
        logits_out = torch.empty(base_logits.shape, dtype=base_logits.dtype, device=dev)
    elif logits_out.shape != base_logits.shape or logits_out.dtype != base_logits.dtype or not logits_out.is_contiguous():
        raise ValueError("logits_out must be a contiguous tensor shaped and typed like base_logits")
    if B == 0 or M == 0:
        return tokens_out, logits_out
    base = base_logits.contiguous()
    first = first_prev_token_ids.to(torch.int64).contiguous()
    w1c, w2c = w1.contiguous(), w2.contiguous()
    r = w1.shape[1]
    if workspace is None:
        workspace = Workspace(B, M, V, r, sample=True, device=dev, processed=True)
    st = _call(dev, _lib.load().dspark_markov_sample_block_processed, _ptr(base), tag, _ptr(first), _ptr(w1c), _ptr(w2c),
               wtag, rules, B, M, V, r, T, int(seed) & (2**64 - 1), int(position_offset), int(batch_offset),
               _ptr(tokens_out), _ptr(logits_out), workspace.ptr, workspace.nbytes)
    _lib.check(st, "sample_block_tokens_processed")
    if check:
        read_device_error(workspace)
    return tokens_out, logits_out
