"""GPU: silu and gelu of the largest finite values, and their derivatives from checkpoints of such values.

An encoded value stands for value (1 +- 2^-4), and for value + 2^-10 of the scale at most where it is smaller than the codes reach; the
functions themselves are some ulp of float32 (2^-18) off.  Beyond |u| = 200 silu and gelu are u or 0 and their derivatives 1 or 0 to
float32's digits.
"""

import numpy as np
import pytest

import oracle.linear8 as ol
import tests.test_gpu_linear8 as base
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

FAR = [200.0, 1e10, 1e30, 2.35e38, 2.37e38, 3.0e38, 3.38e38, float(np.finfo(np.float32).max)]


def _rows(dtype):
    """Each far value in a block of its own, with its negative, with small values, and both together."""
    import torch
    top = float(torch.finfo(base._type(dtype)).max)
    rows = []
    for v in FAR + [top]:
        v = min(v, top)
        for pair in ((v, 0.0), (-v, 0.0), (-v, 1.0), (v, -v)):
            rows.append([0.0] * 3 + list(pair) + [-0.5] + [0.0] * 124)
    return torch.tensor(rows, dtype=torch.float32).to(base._type(dtype))


def _meant(q):
    codes, byte = (base._codes(t) for t in q.unpadded())
    return ol.decode(codes, byte), np.repeat(2.0 ** (byte.astype(np.float64) - 127), 128, axis=1)[:, :q.dim]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32", "fp16"])
def test_encode_after_the_function(kind, dtype):
    import muon_optimizer_step_amd as ms
    x = _rows(dtype)
    gu.say(f"[far] encode {kind} {dtype}")
    r = ms.act8_encode(x.cuda(), activation=kind)
    base._same_codes(r.checkpoint, ol.encode(base._f64(x)), "x")
    got, scale = _meant(r.out)
    with np.errstate(over="ignore"):
        want = ol.act(base._f64(x), kind)
    assert np.isfinite(want).all() and np.isfinite(got).all(), f"NaN codes: {np.argwhere(~np.isfinite(got)).tolist()}"
    assert (np.abs(got - want) <= (2.0 ** -4 + 2.0 ** -18) * np.abs(want) + (2.0 ** -10 + 2.0 ** -18) * scale).all()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32", "fp16"])
def test_backward_from_the_checkpoint(kind, dtype):
    """Also where the nearest code stands for 2^128, which float32 does not hold."""
    import torch
    import muon_optimizer_step_amd as ms
    x = _rows(dtype)
    gu.say(f"[far] backward {kind} {dtype}")
    u8 = ms.act8_encode(x.cuda()).checkpoint
    u, _ = _meant(u8)
    with np.errstate(over="ignore"):
        want, terms = ol.slope(u, kind)
    # the terms of gelu and silu are at most 1 + 1.13 in all; far out one is exact and the other zero
    grad = torch.full(x.shape, 0.75, dtype=base._type(dtype), device="cuda")
    r = ms.act8_backward(u8, grad, kind, codes=True)
    got = base._f64(r.grad)
    assert np.isfinite(got).all(), f"not finite: {np.argwhere(~np.isfinite(got)).tolist()}"
    assert (np.abs(got - 0.75 * want) <= base.U[dtype] * np.abs(want) + 2.0 ** -20 * np.minimum(terms, 3.0) + base.TINY[dtype]).all()
    assert np.isfinite(_meant(r.grad8)[0]).all()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward_with_any_scale(kind):
    """Scales beyond those of the encoding: derivatives of 1 and 0, and of zero codes; NaN codes stay NaN."""
    import torch
    import muon_optimizer_step_amd as ms
    x = torch.zeros(2, 130)
    x[:, 0], x[:, 1], x[:, 3], x[:, 129] = 448.0, -448.0, float("nan"), 2.0 ** -9
    q = ms.act8_encode(x.cuda()).checkpoint
    for scale in (232, 240, 241, 247, 254):
        got = ms.act8_backward(ms.Activation8(q.codes, torch.full_like(q.scale, scale), 130), torch.ones(2, 130, device="cuda"), kind).grad.cpu()
        assert (got[:, 0] == 1).all() and (got[:, 1] == 0).all() and torch.isnan(got[:, 3]).all()
        assert (got[:, 2] == 0.5).all() and (got[:, 4:129] == 0.5).all() and (got[:, 129] == 1).all(), scale


@pytest.mark.parametrize("kind", ["silu", "gelu", "relu2"])
def test_values_that_are_not_finite(kind):
    """NaN is NaN; what the functions make of infinities is not finite, or zero."""
    import torch
    import muon_optimizer_step_amd as ms
    x = torch.ones(3, 128)
    x[0, 5], x[1, 5], x[2, 5] = float("nan"), float("inf"), float("-inf")
    r = ms.act8_encode(x.cuda(), activation=kind)
    nan = (base._codes(r.out.codes) & 0x7F) == 0x7F
    assert nan[0, 5] and nan[1, 5] and nan[:2].sum() == 2 and (nan[2].sum() == nan[2, 5])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_relu2_backward_of_far_values(dtype):
    """2 u is beyond float32 from 1.7e38 on, and u is where its code stands for 2^128; their products with a small gradient, and with
    zero, are not."""
    import torch
    import muon_optimizer_step_amd as ms
    x = _rows(dtype)
    gu.say(f"[far] backward relu2 {dtype}")
    u8 = ms.act8_encode(x.cuda()).checkpoint
    u, _ = _meant(u8)
    assert u.max() == 2.0 ** 128
    for value in (0.0, 2.0 ** -20, -2.0 ** -100):
        grad = torch.full(x.shape, value, dtype=base._type(dtype), device="cuda")
        r = ms.act8_backward(u8, grad, "relu2", codes=True)
        want = value * 2 * np.maximum(u, 0)
        got = base._f64(r.grad)
        assert np.isfinite(got).all(), f"{value}: {np.argwhere(~np.isfinite(got)).tolist()}"
        assert (np.abs(got - want) <= (base.U[dtype] + 2.0 ** -20) * np.abs(want) + base.TINY[dtype]).all(), value
        values, scale = _meant(r.grad8)
        assert (np.abs(values - want) <= (2.0 ** -4 + 2.0 ** -18) * np.abs(want) + (2.0 ** -10 + 2.0 ** -18) * scale).all(), value
    nan = torch.full((1, 128), float("nan"), device="cuda")
    bad = ms.act8_backward(ms.act8_encode(nan).checkpoint, torch.zeros(1, 128, device="cuda"), "relu2", codes=True)
    assert torch.isnan(bad.grad).all() and ((base._codes(bad.grad8.codes) & 0x7F) == 0x7F).all()


def test_relu2_backward_with_any_scale():
    """448 2^(scale - 127) and 2^-9 of it, times 2 and a gradient that brings the product back: exact."""
    import torch
    import muon_optimizer_step_amd as ms
    x = torch.zeros(2, 130)
    x[:, 0], x[:, 1], x[:, 3], x[:, 4] = 448.0, -448.0, float("nan"), 2.0 ** -9
    q = ms.act8_encode(x.cuda()).checkpoint
    for scale in (1, 10, 127, 239, 240, 241, 247, 254):
        u8 = ms.Activation8(q.codes, torch.full_like(q.scale, scale), 130)
        power = max(-126, 127 - scale - 9)
        got = ms.act8_backward(u8, torch.full((2, 130), 2.0 ** power, device="cuda"), "relu2").grad.cpu().double()
        unit = 2.0 ** (scale - 127 + power + 1)
        assert (got[:, 0] == 448.0 * unit).all() and (got[:, 1] == 0).all() and torch.isnan(got[:, 3]).all(), scale
        assert (got[:, 4] == 2.0 ** -9 * unit).all() and (got[:, 5:] == 0).all(), scale


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_relu2_backward_of_far_gradients(dtype):
    """The largest finite gradient times a small u: exact where both are powers of two but for the gradient's own digits."""
    import torch
    import muon_optimizer_step_amd as ms
    top = torch.finfo(base._type(dtype)).max
    for power in (-2, -30, -100):
        u8 = ms.act8_encode(torch.full((3, 40), 2.0 ** power, device="cuda")).checkpoint
        got = ms.act8_backward(u8, torch.full((3, 40), top, dtype=base._type(dtype), device="cuda"), "relu2").grad
        assert (got.double() == top * 2.0 ** (power + 1)).all(), power
