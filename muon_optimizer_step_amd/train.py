"""torch-facing binding of include/muonstep_train.h: argument marshalling onto the C ABI, nothing else."""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

from . import _lib
from .api import _torch


def _run(entry, args, stream, device):
    """entry(*args, HIP stream) with the tensors' device current: on a torch stream of that device, or on its current one."""
    torch = _torch()
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device.index)
    elif stream.device != device:
        raise ValueError(f"stream of {stream.device}, tensors on {device}")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        rc = entry(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = entry(*args, handle)
    _lib.check(rc)


def _used_on(stream, tensors):
    """Tells the allocator that work on `stream` uses the tensors, which the caller may drop before it has run."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _check(t, name: str, dtypes, numel: Optional[int] = None):
    """A contiguous HIP tensor of one of these dtypes (and this many elements)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a HIP device, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, {numel} wanted")


def _same_device(tensors, what: str):
    """The tensors' common device (None for none)."""
    device = None
    for t in tensors:
        if t is None:
            continue
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError(f"{what}: tensors on {device} and {t.device}")
    return device


# ------------------------------------------------------------- AdamW with 8-bit states

def _blocks(numel: int) -> int:
    return -(-numel // _lib.MUON_ADAMW8_BLOCK)


class AdamW8State:
    """Both AdamW moments of one tensor in 8 bits.

    exp_avg and rms hold one e4m3 code per value (torch.float8_e4m3fn), in units of exp_avg_scale and rms_scale, one
    float32 per 256 consecutive values: the first moment is exp_avg * scale, the square root of the second rms * scale.
    """

    __slots__ = ("exp_avg", "exp_avg_scale", "rms", "rms_scale")

    def __init__(self, exp_avg, exp_avg_scale, rms, rms_scale):
        torch = _torch()
        _check(exp_avg, "exp_avg", (torch.float8_e4m3fn,))
        _check(rms, "rms", (torch.float8_e4m3fn,), exp_avg.numel())
        for t, name in ((exp_avg_scale, "exp_avg_scale"), (rms_scale, "rms_scale")):
            _check(t, name, (torch.float32,), _blocks(exp_avg.numel()))
        _same_device((exp_avg, exp_avg_scale, rms, rms_scale), "AdamW8State")
        self.exp_avg, self.exp_avg_scale, self.rms, self.rms_scale = exp_avg, exp_avg_scale, rms, rms_scale

    @classmethod
    def zeros_like(cls, param) -> "AdamW8State":
        """The state before the first step."""
        torch = _torch()
        codes = [torch.zeros(param.shape, dtype=torch.uint8, device=param.device).view(torch.float8_e4m3fn) for _ in "mv"]
        scales = [torch.zeros(_blocks(param.numel()), dtype=torch.float32, device=param.device) for _ in "mv"]
        return cls(codes[0], scales[0], codes[1], scales[1])

    @classmethod
    def from_moments(cls, exp_avg, exp_avg_sq, stream=None) -> "AdamW8State":
        """The 8-bit state nearest to adamw_step's float32 moments (exp_avg_sq not negative)."""
        torch = _torch()
        _check(exp_avg, "exp_avg", (torch.float32,))
        _check(exp_avg_sq, "exp_avg_sq", (torch.float32,), exp_avg.numel())
        device = _same_device((exp_avg, exp_avg_sq), "from_moments")
        with torch.cuda.stream(stream):
            s = cls.zeros_like(exp_avg)
        _run(_lib.load().adamw8_encode, (
            exp_avg.data_ptr(), exp_avg_sq.data_ptr(), s.exp_avg.data_ptr(), s.exp_avg_scale.data_ptr(),
            s.rms.data_ptr(), s.rms_scale.data_ptr(), exp_avg.numel()), stream, device)
        _used_on(stream, (exp_avg, exp_avg_sq))
        return s

    def moments(self, stream=None):
        """(exp_avg, exp_avg_sq) in float32, as adamw_step keeps them."""
        torch = _torch()
        device = self.exp_avg.device
        with torch.cuda.stream(stream):
            m, v = (torch.empty(self.exp_avg.shape, dtype=torch.float32, device=device) for _ in "mv")
        _run(_lib.load().adamw8_decode, (
            self.exp_avg.data_ptr(), self.exp_avg_scale.data_ptr(), self.rms.data_ptr(), self.rms_scale.data_ptr(),
            m.data_ptr(), v.data_ptr(), m.numel()), stream, device)
        _used_on(stream, (self.exp_avg, self.exp_avg_scale, self.rms, self.rms_scale))
        return m, v


def _adamw8_entries(params, grads, states, emas, copies):
    torch = _torch()
    n = len(params)
    emas = emas if emas is not None else [None] * n
    copies = copies if copies is not None else [None] * n
    for x, name in ((grads, "grads"), (states, "states"), (emas, "emas"), (copies, "copies")):
        if len(x) != n:
            raise ValueError(f"{name} must have one entry per parameter")
    fp32 = (torch.float32,)
    entries, seen = [], []
    for i, (p, g, s, e, c) in enumerate(zip(params, grads, states, emas, copies)):
        _check(p, f"params[{i}]", fp32)
        _check(g, f"grads[{i}]", (torch.float32, torch.bfloat16), p.numel())
        if isinstance(s, AdamW8State):
            if s.exp_avg.numel() != p.numel():
                raise ValueError(f"states[{i}] has {s.exp_avg.numel()} elements, params[{i}] {p.numel()}")
            state = (s.exp_avg, s.exp_avg_scale, s.rms, s.rms_scale)
        else:
            try:
                m, v = s
            except (TypeError, ValueError):
                raise TypeError(f"states[{i}] must be an AdamW8State or a pair (exp_avg, exp_avg_sq)") from None
            _check(m, f"states[{i}][0]", fp32, p.numel())
            _check(v, f"states[{i}][1]", fp32, p.numel())
            state = (m, None, v, None)
        if e is not None:
            _check(e, f"emas[{i}]", fp32, p.numel())
        if c is not None:
            _check(c, f"copies[{i}]", (torch.bfloat16,), p.numel())
        tensors = (p, g, *state, e, c)
        seen.extend(tensors)
        entries.append(tuple(t.data_ptr() if t is not None else 0 for t in tensors)
                       + (p.numel(), int(g.dtype == torch.bfloat16)))
    return entries, seen, _same_device(seen, "adamw8")


class PreparedAdamW8:
    """adamw8_step with the tensor table marshalled once."""

    def __init__(self, params, grads, states, *, emas=None, copies=None):
        # the tensors themselves: the caller's lists and states may change
        entries, self._keep, self.device = _adamw8_entries(params, grads, states, emas, copies)
        self.n = len(entries)
        self.table = _lib.adamw8_table(entries)

    def __call__(self, *, lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01, step: int,
                 seed: Optional[int] = None, ema_decay: float = 0.0, stream=None) -> None:
        step = int(step)
        if abs(step) >= 1 << 31:
            raise ValueError(f"step = {step} does not fit 32 bits")
        _run(_lib.load().adamw8_step,
             (self.table, self.n, float(lr), float(betas[0]), float(betas[1]), float(eps), float(weight_decay), step,
              float(ema_decay), 0 if seed is None else 1, 0 if seed is None else int(seed) & 0xFFFFFFFFFFFFFFFF),
             stream, self.device)


def adamw8_step(params, grads, states, *, lr: float, betas=(0.9, 0.999), eps: float = 1e-8,
                weight_decay: float = 0.01, step: int, seed: Optional[int] = None, emas=None, ema_decay: float = 0.0,
                copies=None, stream=None) -> None:
    """AdamW over lists of fp32 tensors, each with 8-bit or 32-bit states (params and states updated in place).

    grads: float32 or bfloat16.  states: an AdamW8State per tensor, or a pair (exp_avg, exp_avg_sq) of float32
    tensors.  step counts the AdamW steps including this one (>= 1).  seed: None rounds the 8-bit states to the
    nearest code; an int rounds them stochastically, from (seed, step, the tensor's place in the list, the value's
    index); a captured graph repeats the step and seed that were captured.  emas: optional list of float32 tensors (or None entries) advanced as ema = d*ema + (1-d)*param' with
    d = ema_decay.  copies: optional list of bfloat16 tensors (or None entries) that receive the updated parameter.
    """
    call = PreparedAdamW8(params, grads, states, emas=emas, copies=copies)
    call(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, step=step, seed=seed, ema_decay=ema_decay, stream=stream)
    _used_on(stream, call._keep)


# ------------------------------------------------------------- loss of the language-model head

class LinearCrossEntropy(NamedTuple):
    """What the head's loss returns: per-token nll and lse; with gradients also the loss and both gradients.

    None of them is part of an autograd graph, also where hidden or weight require gradients: hand grad_hidden on with
    `output.backward(grad_hidden)` or `torch.autograd.grad(output, inputs, grad_hidden)`, and add grad_weight where it belongs.
    """
    nll: object
    lse: object
    loss: object = None
    grad_hidden: object = None
    grad_weight: object = None


def _check_rows(t, name: str, dtype=None, shape=None):
    """A 2-D HIP tensor of a 16-bit float type with contiguous rows."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (torch.bfloat16, torch.float16) or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be {dtype if dtype is not None else 'bfloat16 or float16'}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a HIP device, got {t.device}")
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must be 2-D{f' of shape {tuple(shape)}' if shape is not None else ''}, got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows, strides {t.stride()}")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}'s rows overlap, strides {t.stride()}")


def _check_workspace(t, device):
    """A contiguous tensor of any type on the call's device: the library writes to it."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"workspace must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")


class PreparedLinearCrossEntropy:
    """The head's loss with the tensors marshalled once (same tensors and result buffers every call).

    hidden [tokens, dim] and weight [vocab, dim] (bfloat16 or float16, rows may be strided), targets [tokens] int64.
    grads: compute the loss and the gradients, not only nll and lse (grad_hidden=False or grad_weight=False leaves
    that one out; a tensor given there receives it).  token_weights: float32 [tokens], or None for the mean over the
    tokens whose target is not ignore_index.  softcap: logits are softcap * tanh(z / softcap), 0 for none.
    Each call returns the same LinearCrossEntropy of result tensors, overwritten.
    stream: whose memory the results and the workspace are (None: the current one).  Calls on another one, and from
    another thread, have to be ordered with those before and with the use of the results.
    """

    def __init__(self, hidden, weight, targets, *, token_weights=None, ignore_index: int = -100, softcap: float = 0.0,
                 grads: bool = False, grad_hidden=None, grad_weight=None, workspace=None, stream=None):
        torch = _torch()
        _check_rows(hidden, "hidden")
        _check_rows(weight, "weight", hidden.dtype)
        tokens, dim = hidden.shape
        vocab = weight.shape[0]
        if weight.shape[1] != dim:
            raise ValueError(f"weight has {weight.shape[1]} columns, hidden {dim}")
        _check(targets, "targets", (torch.int64,), tokens)
        if token_weights is not None:
            _check(token_weights, "token_weights", (torch.float32,), tokens)
        if not grads and (token_weights is not None or grad_hidden is not None or grad_weight is not None):
            raise ValueError("token_weights, grad_hidden and grad_weight are for grads=True")
        device = _same_device((hidden, weight, targets, token_weights), "linear_cross_entropy")
        s = stream if stream is not None else torch.cuda.current_stream(device)
        with torch.cuda.stream(s):
            nll, lse = (torch.empty(tokens, dtype=torch.float32, device=device) for _ in "nl")
            loss = torch.empty((), dtype=torch.float32, device=device) if grads else None
            if grads and grad_hidden is None:
                grad_hidden = torch.empty(tokens, dim, dtype=hidden.dtype, device=device)
            if grads and grad_weight is None:
                grad_weight = torch.empty(vocab, dim, dtype=hidden.dtype, device=device)
        grad_hidden = grad_hidden if grad_hidden is not False else None
        grad_weight = grad_weight if grad_weight is not False else None
        if grad_hidden is not None:
            _check_rows(grad_hidden, "grad_hidden", hidden.dtype, (tokens, dim))
        if grad_weight is not None:
            _check_rows(grad_weight, "grad_weight", hidden.dtype, (vocab, dim))
        _same_device((hidden, grad_hidden, grad_weight), "linear_cross_entropy")
        self.result = LinearCrossEntropy(nll, lse, loss, grad_hidden, grad_weight)
        self._keep = (hidden, weight, targets, token_weights, grad_hidden, grad_weight, workspace)
        ptr = lambda t: t.data_ptr() if t is not None else 0  # noqa: E731
        # a single row has no row stride, whatever its tensor says
        pitch = lambda t: t.stride(0) if t is not None and t.shape[0] > 1 else dim  # noqa: E731
        self.problem = _lib.HeadLoss(
            ptr(hidden), ptr(weight), ptr(targets), ptr(token_weights), ptr(loss), ptr(nll), ptr(lse), ptr(grad_hidden),
            ptr(grad_weight), tokens, vocab, dim, pitch(hidden), pitch(weight), pitch(grad_hidden), pitch(grad_weight),
            int(ignore_index), float(softcap),
            _lib.MUON_HEAD_BF16 if hidden.dtype == torch.bfloat16 else _lib.MUON_HEAD_FP16)
        self._lib = _lib.load()
        need = self._lib.head_loss_workspace_size(self.problem)
        if need == 0:
            raise _lib.MuonError(_lib.MUON_ERR_INVALID_ARG, self._lib.muon_last_error().decode())
        if workspace is None:
            # allocated on the stream the calls run on, so that its memory is reused only in that stream's order
            with torch.cuda.stream(s):
                workspace = torch.empty(int(need), dtype=torch.uint8, device=device)
        _check_workspace(workspace, device)
        self.workspace = workspace
        self._ws = (workspace.data_ptr(), workspace.numel() * workspace.element_size())
        self.device = device

    def __call__(self, stream=None) -> LinearCrossEntropy:
        _run(self._lib.head_loss, (self.problem, *self._ws), stream, self.device)
        return self.result


def _once(hidden, weight, targets, stream, **kw):
    call = PreparedLinearCrossEntropy(hidden, weight, targets, stream=stream, **kw)
    result = call(stream)
    _used_on(stream, call._keep)
    return result


def linear_cross_entropy(hidden, weight, targets, *, ignore_index: int = -100, softcap: float = 0.0, workspace=None,
                         stream=None) -> LinearCrossEntropy:
    """Scores tokens: nll and log-sum-exp of each under softmax(hidden @ weight.T), float32, without the logits.

    workspace: None takes one for this call from the stream's memory (calls from several threads, and calls captured in
    a graph, do not share any).
    """
    return _once(hidden, weight, targets, stream, ignore_index=ignore_index, softcap=softcap, workspace=workspace)


def linear_cross_entropy_grad(hidden, weight, targets, *, token_weights=None, ignore_index: int = -100,
                              softcap: float = 0.0, grad_hidden=None, grad_weight=None, workspace=None,
                              stream=None) -> LinearCrossEntropy:
    """The loss of a training step with the gradients of hidden and weight (see PreparedLinearCrossEntropy).

    workspace: as in linear_cross_entropy.
    """
    return _once(hidden, weight, targets, stream, token_weights=token_weights, ignore_index=ignore_index, softcap=softcap,
                 grads=True, grad_hidden=grad_hidden, grad_weight=grad_weight, workspace=workspace)
