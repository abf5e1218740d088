"""GPU: matmul8 with exact products against 64 bits.

Tolerances, from the arithmetic.  Decoded codes multiply without rounding.  A block of 128 products is summed in float32 by the
16-bit matrix instruction, at most 128 additions each off by 2^-23 of the magnitudes (it may cut rather than round); the block's sum is
scaled by a power of two, exactly; dim / 128 such sums are added, and up to 64 parts of K joined, 2^-24 each:
(dim / 128 + 200) 2^-23 of the sum of magnitudes covers them.  Then one rounding to a 16-bit type.
"""

import numpy as np
import pytest

import tests.test_gpu_linear8 as base
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


def _product(rows, cols, dim, dtype, seed=0, **kw):
    import torch
    import muon_optimizer_step_amd as ms
    a8 = ms.act8_encode(torch.from_numpy(base._values(rows, dim, seed + 1)).cuda()).checkpoint
    b8 = ms.weight8_encode(torch.from_numpy(base._values(cols, dim, seed + 2, 0.3)).cuda())
    y = ms.matmul8(a8, b8, dtype=base._type(dtype), exact=True, **kw)
    a, b = base._f64(a8.decode(torch.float32)), base._f64(b8.decode(torch.float32))
    return y, a, b


def _check(y, a, b, dtype, label):
    want = a @ b.T
    tol = (a.shape[1] / 128 + 200) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T) * (1 + base.U[dtype]) + base.U[dtype] * np.abs(want) + base.TINY[dtype]
    err = np.abs(base._f64(y) - want)
    assert (err <= tol).all(), f"{label}: worst {np.nanmax(err / tol):.3g} of the tolerance"


# rows, cols, dim: single rows and columns, both tiles, ends inside tiles, blocks, stages and chunks of 16, K split, over 16 stages
SIZES = [(1, 1, 1), (1, 4096, 1024), (2, 33, 15), (16, 257, 2200), (17, 64, 129), (31, 31, 255), (33, 130, 600), (64, 300, 16),
         (65, 8, 2304), (128, 128, 128), (129, 255, 1000), (200, 520, 4500), (700, 1100, 640), (20, 70, 66000), (1025, 2050, 2300),
         (2050, 2100, 300), (5000, 300, 200), (3000, 2500, 2600)]


@pytest.mark.parametrize("rows,cols,dim", SIZES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_exact_matmul(rows, cols, dim, dtype):
    gu.say(f"[matmul8 exact] {rows} x {cols} x {dim} {dtype}")
    y, a, b = _product(rows, cols, dim, dtype)
    assert y.dtype == base._type(dtype) and tuple(y.shape) == (rows, cols)
    _check(y, a, b, dtype, "matmul8")


@pytest.mark.parametrize("rows,cols,dim", [(5, 64, 512), (64, 512, 2048), (300, 500, 1000), (2050, 2100, 700)])
def test_error_in_norm(rows, cols, dim):
    """float32's digits: the 8-bit unit's sums are 2.6e-5 off."""
    y, a, b = _product(rows, cols, dim, "fp32")
    assert gu.rel_frob(base._f64(y), a @ b.T) <= 2.0 ** -20


def test_sums_that_cancel():
    """256 - 256 + 2^-9, in one group of 8 products: the small one is all that is left."""
    import torch
    import muon_optimizer_step_amd as ms
    for rows in (3, 200):
        x = torch.zeros(rows, 130)
        x[:, 0], x[:, 1], x[:, 2] = 16.0, 16.0, 2.0 ** -4
        w = torch.zeros(5, 130)
        w[:, 0], w[:, 1], w[:, 2] = 16.0, -16.0, 2.0 ** -5
        y = ms.matmul8(ms.act8_encode(x.cuda()).checkpoint, ms.weight8_encode(w.cuda()), dtype=torch.float32, exact=True)
        assert (y == 2.0 ** -9).all()


@pytest.mark.parametrize("rows", [3, 40, 1500])
def test_nan_stays_in_its_row_and_column(rows):
    import torch
    import muon_optimizer_step_amd as ms
    x, w = torch.from_numpy(base._values(rows, 300, 1)), torch.from_numpy(base._values(1400, 300, 2))
    x[1, 7], w[130, 299] = float("inf"), float("nan")
    y = base._f64(ms.matmul8(ms.act8_encode(x.cuda()).checkpoint, ms.weight8_encode(w.cuda()), dtype=torch.float32, exact=True))
    bad = np.isnan(y)
    assert bad[1].all() and bad[:, 130].all() and bad.sum() == rows + 1400 - 1


@pytest.mark.parametrize("rows,cols", [(5, 77), (70, 1030), (1500, 1501)])
def test_into_strided_rows(rows, cols):
    """A slice of a wider float32 output, off the 16-byte grid, and what lies around it untouched."""
    import torch
    import muon_optimizer_step_amd as ms
    a8 = ms.act8_encode(torch.from_numpy(base._values(rows, 1150, 1)).cuda()).checkpoint
    b8 = ms.weight8_encode(torch.from_numpy(base._values(cols, 1150, 2)).cuda())
    want = ms.PreparedMatmul8(a8, b8, dtype=torch.float32)()
    for pitch, off in ((cols + 19, 0), (cols + 24, 3)):
        flat = torch.full((rows * pitch + off + 8,), 7.0, device="cuda")
        view = flat[off:off + rows * pitch].view(rows, pitch)[:, :cols]
        assert ms.matmul8(a8, b8, out=view, exact=True) is view
        assert torch.equal(view, want)
        view.fill_(7.0)
        assert (flat == 7.0).all()


@pytest.mark.parametrize("scale,power", [(1, 100), (10, 110), (127, 0), (230, -100), (254, -100)])
def test_any_scale(scale, power):
    import torch
    import muon_optimizer_step_amd as ms
    for rows in (4, 90, 1500):
        q = ms.act8_encode(torch.ones(rows, 130, device="cuda")).checkpoint
        a8 = ms.Activation8(q.codes, torch.full_like(q.scale, scale), 130)
        w = torch.zeros(1400, 130)
        w[:, 129] = 2.0 ** power
        y = ms.matmul8(a8, ms.weight8_encode(w.cuda()), dtype=torch.float32, exact=True)
        assert (base._f64(y) == 256.0 * 2.0 ** (scale - 127 + power)).all()


def test_which_results_are_exact():
    """A prepared call has exact products for float32 results, and elsewhere where it is told; a one-shot call is told."""
    import torch
    import muon_optimizer_step_amd as ms
    a8 = ms.act8_encode(torch.from_numpy(base._values(300, 1000, 1)).cuda()).checkpoint
    b8 = ms.weight8_encode(torch.from_numpy(base._values(200, 1000, 2)).cuda())
    exact = ms.matmul8(a8, b8, dtype=torch.float32, exact=True)
    assert torch.equal(ms.PreparedMatmul8(a8, b8, dtype=torch.float32)(), exact)
    assert torch.equal(ms.PreparedMatmul8(a8, b8, out=torch.empty_like(exact))(), exact)
    assert torch.equal(ms.PreparedMatmul8(a8, b8, exact=True)(), exact.bfloat16())
    assert torch.equal(ms.PreparedMatmul8(a8, b8)(), ms.matmul8(a8, b8))
    for make in (ms.PreparedMatmul8, ms.matmul8):
        with pytest.raises(TypeError, match="exact=True"):
            make(a8, b8, dtype=torch.float32, exact=False)
        with pytest.raises(TypeError, match="float64"):
            make(a8, b8, dtype=torch.float64, exact=True)


@pytest.mark.parametrize("rows,cols,dim", [(1, 512, 2048), (64, 256, 8192), (1500, 1400, 600)])
def test_captured_and_replayed(rows, cols, dim):
    import torch
    import muon_optimizer_step_amd as ms
    x, w = torch.empty(rows, dim, device="cuda"), torch.empty(cols, dim, device="cuda")

    def step():
        return ms.matmul8(ms.act8_encode(x).checkpoint, ms.weight8_encode(w), dtype=torch.float32, exact=True)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for seed in range(4):
        x.copy_(torch.from_numpy(base._values(rows, dim, seed)))
        w.copy_(torch.from_numpy(base._values(cols, dim, seed + 9)))
        graph.replay()
        got = y.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, step()), seed


def test_past_32_bits():
    """A float32 result of over 2^32 bytes: its last rows are those of the last rows alone, to the bit where K is not split."""
    import torch
    import muon_optimizer_step_amd as ms
    rows, cols = 270_000, 4100
    x = torch.zeros(rows, 40, dtype=torch.bfloat16, device="cuda")
    x[-300:] = torch.randn(300, 40, device="cuda").bfloat16()
    w8 = ms.weight8_encode(torch.randn(cols, 40, device="cuda"))
    y = ms.matmul8(ms.act8_encode(x).checkpoint, w8, dtype=torch.float32, exact=True)
    assert y.numel() * 4 > 1 << 32
    tail = ms.matmul8(ms.act8_encode(x[-300:]).checkpoint, w8, dtype=torch.float32, exact=True)
    assert torch.equal(y[-300:], tail) and not y[:-300].any() and tail.any()
