"""GPU: the row-wise passes' results in every form in which they are stored, to the bit: large and small, with rows on and off the grids of
16 and 128 bytes, each type and function, against the same call on slices of some rows and against the definition."""

import numpy as np
import pytest

import oracle.linear8 as ol
import tests.test_gpu_linear8 as base
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


def _inputs(rows, dim, dtype, seed=0):
    import torch
    import muon_optimizer_step_amd as ms
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.randn(rows, dim, generator=g, device="cuda") * torch.exp(torch.randn(dim, generator=g, device="cuda"))
    grad = torch.randn(rows, dim, generator=g, device="cuda").to(base._type(dtype))
    return ms.act8_encode(u).checkpoint, grad


def _rows_of(q, a, b):
    import muon_optimizer_step_amd as ms
    return ms.Activation8(q.codes[a:b], q.scale[a:b], q.dim)


# MiB of the result, dim: rows of whole lines, of whole 16 bytes, of neither; below and above what a cache holds
SIZES = [(1, 1024), (1, 1000), (1, 1001), (80, 4096), (80, 1000), (80, 4001), (300, 4096), (300, 1000), (300, 4001)]


@pytest.mark.parametrize("mib,dim", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_backward_of_any_size(mib, dim, dtype):
    import torch
    import muon_optimizer_step_amd as ms
    rows = (mib << 20) // (dim * (4 if dtype == "fp32" else 2)) + 3
    gu.say(f"[stores] backward {rows} x {dim} {dtype}")
    u8, grad = _inputs(rows, dim, dtype)
    step = min(-(-rows // 3), (8 << 20) // dim)
    for kind in ("relu2", "silu", "gelu"):
        alone = ms.act8_backward(u8, grad, kind).grad
        both = ms.act8_backward(u8, grad, kind, codes=True)
        place = grad.clone()
        ms.act8_backward(u8, place, kind, out=place)
        assert torch.equal(both.grad, alone) and torch.equal(place, alone)
        for a in range(0, rows, step):
            b = min(rows, a + step)
            part = ms.act8_backward(_rows_of(u8, a, b), grad[a:b], kind, codes=True)
            assert torch.equal(alone[a:b], part.grad), (kind, a)
            for got, want in zip(_rows_of(both.grad8, a, b).unpadded(), part.grad8.unpadded()):
                assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), (kind, a)
        # first and last rows against the definition
        for sl in (slice(0, 70), slice(rows - 70, rows)):
            u = base._f64(_rows_of(u8, sl.start, sl.stop).decode(torch.float32))
            s, terms = ol.slope(u, kind)
            want = base._f64(grad[sl]) * s
            tol = base.U[dtype] * np.abs(want) + 2.0 ** -20 * np.abs(base._f64(grad[sl])) * terms + base.TINY[dtype]
            assert (np.abs(base._f64(alone[sl]) - want) <= tol).all(), kind


@pytest.mark.parametrize("mib,dim", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_decode_of_any_size(mib, dim, dtype):
    """Exact: codes times powers of two, rounded once."""
    import torch
    rows = (mib << 20) // (dim * (4 if dtype == "fp32" else 2)) + 3
    gu.say(f"[stores] decode {rows} x {dim} {dtype}")
    u8, _ = _inputs(rows, dim, dtype, 1)
    got = u8.decode(base._type(dtype))
    codes, byte = u8.unpadded()
    scale = torch.exp2(byte.float() - 127)
    for a in range(0, rows, 20000):
        wide = scale[a:a + 20000].repeat_interleave(128, dim=1)[:, :dim]
        want = (codes[a:a + 20000].float() * wide).to(base._type(dtype))
        assert torch.equal(got[a:a + 20000], want), a


@pytest.mark.parametrize("off", [0, 8, 3])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_results_between_other_values(off, dtype):
    """A slice of a wider tensor, at 128, 16 and 2 (4) bytes: what lies around it is not touched."""
    import torch
    import muon_optimizer_step_amd as ms
    for rows, dim in ((70, 200), (9000, 4001)):
        u8, grad = _inputs(rows, dim, dtype, 2)
        want = ms.act8_backward(u8, grad, "relu2").grad
        pitch = -(-(dim + off + 1) // 64) * 64
        wide = torch.full((rows, pitch), 7.0, dtype=grad.dtype, device="cuda")
        out = wide[:, off:off + dim]
        assert torch.equal(ms.act8_backward(u8, grad, "relu2", out=out).grad, want)
        out.fill_(7.0)
        assert (wide == 7.0).all()


def test_backward_past_32_bits():
    """The last rows and some in the middle of a result of over 2^32 bytes are those of these rows alone."""
    import torch
    import muon_optimizer_step_amd as ms
    rows, dim = 300_000, 8192
    u8, grad = _inputs(8192, dim, "bf16", 3)
    full = ms.Activation8.empty(rows, dim)
    big = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
    for a in range(0, rows, 8192):
        n = min(8192, rows - a)
        full.codes[a:a + n].view(torch.uint8).copy_(u8.codes[:n].view(torch.uint8))
        full.scale[a:a + n] = u8.scale[:n]
        big[a:a + n] = grad[:n]
    part = ms.act8_backward(u8, grad, "silu", codes=True)
    r = ms.act8_backward(full, big, "silu", out=big, codes=True)
    for a in range(0, rows, 8192):
        n = min(8192, rows - a)
        assert torch.equal(big[a:a + n], part.grad[:n]), a
        for got, want in zip(_rows_of(r.grad8, a, a + n).unpadded(), part.grad8.unpadded()):
            assert torch.equal(got.view(torch.uint8), want[:n].view(torch.uint8)), a
