"""torch-facing binding of include/muonstep_train.h: argument marshalling onto the C ABI, nothing else."""

from __future__ import annotations

import ctypes
from typing import Optional

from . import _lib
from .api import _stream_handle, _torch


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
        _lib.check(_lib.load().adamw8_encode(
            exp_avg.data_ptr(), exp_avg_sq.data_ptr(), s.exp_avg.data_ptr(), s.exp_avg_scale.data_ptr(),
            s.rms.data_ptr(), s.rms_scale.data_ptr(), exp_avg.numel(), _stream_handle(stream, device)))
        return s

    def moments(self, stream=None):
        """(exp_avg, exp_avg_sq) in float32, as adamw_step keeps them."""
        torch = _torch()
        device = self.exp_avg.device
        with torch.cuda.stream(stream):
            m, v = (torch.empty(self.exp_avg.shape, dtype=torch.float32, device=device) for _ in "mv")
        _lib.check(_lib.load().adamw8_decode(
            self.exp_avg.data_ptr(), self.exp_avg_scale.data_ptr(), self.rms.data_ptr(), self.rms_scale.data_ptr(),
            m.data_ptr(), v.data_ptr(), m.numel(), _stream_handle(stream, device)))
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
    return entries, _same_device(seen, "adamw8")


class PreparedAdamW8:
    """adamw8_step with the tensor table marshalled once."""

    def __init__(self, params, grads, states, *, emas=None, copies=None):
        self._keep = (list(params), list(grads), list(states), emas, copies)
        entries, self.device = _adamw8_entries(params, grads, states, emas, copies)
        self.n = len(entries)
        self.table = _lib.adamw8_table(entries)

    def __call__(self, *, lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01, step: int,
                 seed: Optional[int] = None, ema_decay: float = 0.0, stream=None) -> None:
        rc = _lib.load().adamw8_step(self.table, self.n, lr, betas[0], betas[1], eps, weight_decay, step, ema_decay,
                                     0 if seed is None else 1, 0 if seed is None else seed & 0xFFFFFFFFFFFFFFFF,
                                     _stream_handle(stream, self.device))
        _lib.check(rc)


def adamw8_step(params, grads, states, *, lr: float, betas=(0.9, 0.999), eps: float = 1e-8,
                weight_decay: float = 0.01, step: int, seed: Optional[int] = None, emas=None, ema_decay: float = 0.0,
                copies=None, stream=None) -> None:
    """AdamW over lists of fp32 tensors, each with 8-bit or 32-bit states (params and states updated in place).

    grads: float32 or bfloat16.  states: an AdamW8State per tensor, or a pair (exp_avg, exp_avg_sq) of float32
    tensors.  step counts the AdamW steps including this one (>= 1).  seed: None rounds the 8-bit states to the
    nearest code; an int rounds them stochastically, from (seed, step, the tensor's place in the list, the value's
    index).  emas: optional list of float32 tensors (or None entries) advanced as ema = d*ema + (1-d)*param' with
    d = ema_decay.  copies: optional list of bfloat16 tensors (or None entries) that receive the updated parameter.
    """
    PreparedAdamW8(params, grads, states, emas=emas, copies=copies)(
        lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, step=step, seed=seed, ema_decay=ema_decay,
        stream=stream)
