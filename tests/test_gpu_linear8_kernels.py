"""GPU: every kernel of matmul8 and act8_grad_weight, with stages and ends of every kind, against 64 bits.

Which kernel a size goes to is the library's choice; each test says which one it is for and the profiling hook tells which one ran, so
that other choices cannot leave a kernel untested.  Tolerances as in test_gpu_linear8.py; the 64-bit products are computed on the
device.  Blocks of K have unlike scales in both operands, whose products are alike: a scale of another block shows.
"""

import contextlib

import pytest

import tests.test_gpu_linear8 as base
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def _launches():
    """The names of the launches within, in a list that is filled at the end."""
    import muon_optimizer_step_amd as ms
    names = []
    ms.profile_read()
    ms.profile_enable(True)
    try:
        yield names
        names.extend(ms.profile_read())
    finally:
        ms.profile_enable(False)


def _values(rows, dim, seed, block_power=0):
    """Values with rows and columns of unlike size and zeros among them; block b of columns times 2^(block_power e_b)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, dim, generator=g, device="cuda")
    x *= torch.exp(0.3 * torch.randn(dim, generator=g, device="cuda")) * torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    x[torch.rand(rows, dim, generator=g, device="cuda") < 0.05] = 0.0
    blocks = torch.Generator(device="cuda").manual_seed(1234)
    power = torch.randint(-5, 6, (-(-dim // 128),), generator=blocks, device="cuda").repeat_interleave(128)[:dim]
    return x * torch.exp2(block_power * power)


def _wide(q):
    import torch
    return q.decode(torch.float32).double()


def _check(got, want, tol, label):
    err = (got.double() - want).abs_()
    bad = ~(err <= tol)
    assert not bad.any(), f"{label}: {int(bad.sum())} values, worst {float((err / tol).nan_to_num(0).max()):.3g} of the tolerance, first at {bad.nonzero()[0].tolist()}"


def _check_product(y, a, b, dtype, label):
    want = a @ b.t()
    tol = (2.0 ** -10 + (a.shape[1] + 16) * 2.0 ** -23) * (1 + base.U[dtype]) * (a.abs() @ b.abs().t()) + base.U[dtype] * want.abs() + base.TINY[dtype]
    _check(y, want, tol, label)


# kernel, parts of K (True: more than one), rows, cols, dim.  Stages of 128 in all or a part: 1 and up to past a ring's length, 16 (whose scales
# a register holds), 17 and more; whole and ragged tiles, and K that ends on and off chunks of 16 and stages.
PRODUCTS = [
    ("matmul8_rows", False, 1, 8192, 8192), ("matmul8_rows", False, 16, 515, 4099),
    ("matmul8_32", False, 18, 16, 16), ("matmul8_32", False, 17, 16, 139), ("matmul8_32", False, 19, 16, 2146),
    ("matmul8_32", False, 4144, 16, 4676),
    ("matmul8_64", False, 4399, 36, 16), ("matmul8_64", False, 33, 4150, 140), ("matmul8_64", False, 4266, 35, 260),
    ("matmul8_64", False, 64, 8192, 500), ("matmul8_64", False, 64, 8192, 520), ("matmul8_64", False, 64, 8192, 650),
    ("matmul8_64", False, 64, 8192, 777), ("matmul8_64", False, 64, 8192, 900), ("matmul8_64", False, 4550, 33, 1993),
    ("matmul8_64", False, 33, 4154, 2071), ("matmul8_64", False, 36, 4331, 2375), ("matmul8_64", False, 3047, 69, 4224),
    ("matmul8_64", True, 17, 16, 3059), ("matmul8_64", True, 17, 2342, 6198), ("matmul8_64", True, 4283, 16, 5702),
    ("matmul8_64", True, 300, 300, 30000),
    ("matmul8_128", False, 5514, 135, 16), ("matmul8_128", False, 654, 3100, 129), ("matmul8_128", False, 344, 5559, 268),
    ("matmul8_128", False, 2048, 2048, 512), ("matmul8_128", False, 1025, 2050, 1930), ("matmul8_128", False, 388, 4706, 2084),
    ("matmul8_128", False, 1025, 2050, 2300), ("matmul8_128", False, 335, 5477, 4275),
    ("matmul8_128", True, 4333, 16, 6488), ("matmul8_128", True, 4144, 66, 7776), ("matmul8_128", True, 5536, 145, 4317),
    ("matmul8_128", True, 520, 520, 16000),
    ("matmul8_256", False, 3486, 3542, 257), ("matmul8_256", False, 49995, 4003, 307), ("matmul8_256", False, 3900, 4000, 385),
    ("matmul8_256", False, 3840, 4096, 640), ("matmul8_256", False, 4096, 4096, 2048), ("matmul8_256", False, 8045, 1552, 1945),
    ("matmul8_256", False, 1420, 5599, 2092), ("matmul8_256", False, 3345, 2359, 2208), ("matmul8_256", False, 1030, 7336, 4226),
    ("matmul8_256", False, 262, 27196, 5142),
]


@pytest.mark.parametrize("kernel,parts,rows,cols,dim", PRODUCTS)
def test_matmul(kernel, parts, rows, cols, dim):
    import torch
    import muon_optimizer_step_amd as ms
    gu.say(f"[kernels] {kernel} {rows} x {cols} x {dim}")
    a8 = ms.act8_encode(_values(rows, dim, rows + 1, 1)).checkpoint
    b8 = ms.weight8_encode(_values(cols, dim, cols + 2, -1))
    a, b = _wide(a8), _wide(b8)
    for dtype in ("bf16", "fp16"):
        with _launches() as names:
            y = ms.matmul8(a8, b8, dtype=base._type(dtype))
        assert sorted(names) == sorted([kernel] + ["matmul8_join"] * parts)
        _check_product(y, a, b, dtype, f"{kernel} {dtype}")
        assert torch.equal(ms.matmul8(a8, b8, dtype=base._type(dtype)), y)
    # the 64-bit product of a few rows on the host, which shares nothing with the device's
    some = [0, rows // 2, rows - 1]
    assert gu.rel_frob((a[some] @ b.t()).cpu().numpy(), a[some].cpu().numpy() @ b.cpu().numpy().T) < 1e-13


@pytest.mark.parametrize("kernel,rows,cols,dim", [("matmul8_32", 40, 200, 300), ("matmul8_64", 64, 8192, 520), ("matmul8_64", 36, 4331, 2375),
                                                  ("matmul8_128", 1025, 2050, 2300), ("matmul8_256", 3486, 3542, 300),
                                                  ("matmul8_256", 1420, 5599, 2092)])
def test_matmul_nan_stays_in_its_row_and_column(kernel, rows, cols, dim):
    """NaN in the last stage, where the chunks behind K's end repeat its first one, and in the last row and column."""
    import torch
    import muon_optimizer_step_amd as ms
    x, w = _values(rows, dim, 1), _values(cols, dim, 2)
    last = (dim - 1) // 128 * 128
    for at in (last, min(last + 17, dim - 1), dim - 1, 5):
        for row, col in ((rows - 1, 3), (rows // 2, cols - 1)):
            p, q = x.clone(), w.clone()
            p[row, at], q[col, at] = float("nan"), float("inf")
            with _launches() as names:
                y = ms.matmul8(ms.act8_encode(p).checkpoint, ms.weight8_encode(q))
            assert kernel in names
            bad = torch.isnan(y)
            assert bad[row].all() and bad[:, col].all() and int(bad.sum()) == rows + cols - 1, (at, row, col)


@pytest.mark.parametrize("kernel,rows,cols,dim", [("matmul8_64", 4266, 35, 260), ("matmul8_64", 36, 4331, 2375), ("matmul8_128", 1025, 2050, 1930),
                                                  ("matmul8_256", 3486, 3542, 257)])
def test_matmul_into_strided_rows(kernel, rows, cols, dim):
    """Slices of a wider y on the grids of 128, 16 and 2 bytes; what lies around them is not touched."""
    import torch
    import muon_optimizer_step_amd as ms
    a8, b8 = ms.act8_encode(_values(rows, dim, 1)).checkpoint, ms.weight8_encode(_values(cols, dim, 2))
    want = ms.matmul8(a8, b8)
    for pitch, off in ((-(-cols // 64) * 64 + 64, 0), (-(-cols // 64) * 64 + 8, 8), (cols + 5, 3)):
        flat = torch.full((rows * pitch + off + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
        view = flat[off:off + rows * pitch].view(rows, pitch)[:, :cols]
        with _launches() as names:
            ms.matmul8(a8, b8, out=view)
        assert kernel in names and torch.equal(view, want)
        view.fill_(7.0)
        assert (flat == 7.0).all()


@pytest.mark.parametrize("kernel,rows,cols", [("matmul8_64", 64, 8192), ("matmul8_128", 1025, 2050), ("matmul8_256", 3486, 3542)])
@pytest.mark.parametrize("scale,power", [(1, 100), (127, 0), (254, -100)])
def test_matmul_takes_any_scale(kernel, rows, cols, scale, power):
    import torch
    import muon_optimizer_step_amd as ms
    q = ms.act8_encode(torch.ones(rows, 390, device="cuda")).checkpoint
    a8 = ms.Activation8(q.codes, torch.full_like(q.scale, scale), 390)
    w = torch.zeros(cols, 390, device="cuda")
    w[:, 389] = 2.0 ** power
    with _launches() as names:
        y = ms.matmul8(a8, ms.weight8_encode(w))
    assert kernel in names and (y.double() == 256.0 * 2.0 ** (scale - 127 + power)).all()


# ------------------------------------------------------------- the weight's gradient

# kernel, parts, rows, cols, dim.  Stages of 64 rows: 1 to 6 and more for each tile, 40 to 65 for the deep form (whose loop takes 4 at a time)
GRADS = [
    ("act8_grad_128", False, 40, 16, 16), ("act8_grad_128", False, 100, 70, 300), ("act8_grad_128", True, 16384, 512, 512),
    ("act8_grad_256", False, 16, 13102, 567), ("act8_grad_256", False, 66, 525, 13195), ("act8_grad_256", False, 133, 14750, 521),
    ("act8_grad_256", False, 195, 646, 11199), ("act8_grad_256", False, 260, 646, 11199), ("act8_grad_256", False, 330, 646, 11199),
    ("act8_grad_256", False, 700, 4090, 2500), ("act8_grad_256", False, 900, 3000, 3000), ("act8_grad_256", True, 3000, 2049, 2047),
    ("act8_grad_256", True, 4875, 8426, 137), ("act8_grad_256", True, 16384, 4096, 1024),
    ("act8_grad_128_deep", False, 2516, 131, 8520), ("act8_grad_128_deep", False, 2600, 131, 8520),
    ("act8_grad_128_deep", False, 2625, 1500, 1700), ("act8_grad_128_deep", False, 2690, 1500, 1700),
    ("act8_grad_128_deep", False, 2760, 1500, 1700), ("act8_grad_128_deep", False, 4096, 2048, 2048),
    ("act8_grad_128_deep", True, 10163, 18, 5688), ("act8_grad_128_deep", True, 16400, 2048, 500),
]


def _grad_inputs(rows, cols, dim):
    import muon_optimizer_step_amd as ms
    x8 = ms.act8_encode(_values(rows, dim, rows + 1, 1)).checkpoint
    return x8, _values(rows, cols, cols + 2).bfloat16()


@pytest.mark.parametrize("kernel,parts,rows,cols,dim", GRADS)
def test_grad_weight(kernel, parts, rows, cols, dim):
    import torch
    import muon_optimizer_step_amd as ms
    gu.say(f"[kernels] {kernel} {rows} x {cols} x {dim}")
    x8, grad = _grad_inputs(rows, cols, dim)
    x, g = _wide(x8), grad.double()
    sums, mags = g.t().contiguous() @ x, g.abs().t().contiguous() @ x.abs()
    launches = [kernel] + ["act8_grad_join"] * parts + ["act8_grad_pack"] * (cols % 8 != 0)
    with _launches() as names:
        got = ms.act8_grad_weight(x8, grad)
    assert sorted(names) == sorted(launches)
    bound = (rows + 48) * 2.0 ** -23
    _check(got, sums, bound * mags + 1e-37, kernel)
    assert torch.equal(ms.act8_grad_weight(x8, grad), got)
    before = _values(cols, dim, 5) * float(mags.mean())
    out = before.clone()
    with _launches() as names:
        ms.act8_grad_weight(x8, grad, out=out, accumulate=True)
    assert sorted(names) == sorted(launches)
    _check(out, sums + before.double(), bound * (mags + before.double().abs()) + 1e-37, f"{kernel}, added")


@pytest.mark.parametrize("kernel,rows,cols,dim", [("act8_grad_128", 100, 70, 300), ("act8_grad_256", 700, 4090, 2500),
                                                  ("act8_grad_256", 195, 646, 11199), ("act8_grad_128_deep", 2625, 1500, 1700)])
def test_grad_weight_strides(kernel, rows, cols, dim):
    """A gradient in a wider tensor of NaN, into slices on and off the 16-byte grid; nothing around them is touched."""
    import torch
    import muon_optimizer_step_amd as ms
    x8, grad = _grad_inputs(rows, cols, dim)
    want = ms.act8_grad_weight(x8, grad)
    for wider, off, at in ((24, 8, 0), (7, 3, 4), (-(-cols // 8) * 8 - cols + 8, 0, 3)):
        room = torch.full((rows, cols + wider + off), float("nan"), dtype=torch.bfloat16, device="cuda")
        view = room[:, off:off + cols]
        view.copy_(grad)
        wide = torch.full((cols, -(-(dim + at) // 4) * 4 + 4), 5.0, device="cuda")
        out = wide[:, at:at + dim]
        with _launches() as names:
            ms.act8_grad_weight(x8, view, out=out)
        assert kernel in names and torch.equal(out, want), (wider, off, at)
        out.fill_(5.0)
        assert (wide == 5.0).all()


@pytest.mark.parametrize("kernel,rows,cols,dim", [("act8_grad_128", 100, 70, 300), ("act8_grad_256", 133, 14750, 521),
                                                  ("act8_grad_256", 700, 4096, 2500), ("act8_grad_128_deep", 2625, 1500, 1700)])
def test_grad_weight_infinities_stay_where_they_belong(kernel, rows, cols, dim):
    """An infinite gradient of the last row, and a NaN of x there: rows behind it are none."""
    import torch
    import muon_optimizer_step_amd as ms
    x, grad = torch.ones(rows, dim, device="cuda"), torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    grad[-1, 5], grad[-1, cols - 1] = float("inf"), float("-inf")
    x[-1, 7], x[-1, dim - 1] = -1.0, float("nan")
    with _launches() as names:
        got = ms.act8_grad_weight(ms.act8_encode(x).checkpoint, grad)
    assert kernel in names
    want = torch.full((cols, dim), float(rows), device="cuda")
    want[:, 7] -= 2.0
    want[5], want[cols - 1] = float("inf"), float("-inf")
    want[5, 7], want[cols - 1, 7] = float("-inf"), float("inf")
    want[:, dim - 1] = float("nan")
    assert torch.equal(got.nan_to_num(nan=1e9), want.nan_to_num(nan=1e9))
