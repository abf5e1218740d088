"""GPU: linear layers in 8 bits against the float64 oracle.

Tolerances, from the arithmetic:
* codes and scales are defined to the bit: a scale comes from the bits of a block's largest value, and value / scale is
  exact.  relu2's u^2 has one rounding in float32, which the oracle makes too; silu and gelu are a few ulp of float32 off,
  so their codes stand for the value to half a step of e4m3 (2^-4 of it, or half the smallest step, 2^-10 of the scale),
  and their scales may be a neighbour's where the block's largest value is at the border;
* matmul8: the matrix unit adds 8 products at a time, each cut to 2^-13 of the largest of the 8 (measured: 16 x 16 + 2^-5
  is exact, 2^-6 is lost), so 7 of 8 lose up to 7 x 2^-13 < 2^-10 of the sum of magnitudes together; the sums themselves are in
  float32, (K + 16) 2^-23 of it; then one rounding to the output's type, u = 2^-8 of it in bf16, 2^-11 in fp16;
* the weight's gradient sums exact 16-bit products in float32: (K + 48) 2^-23 of the sum of magnitudes (the matrix unit may
  cut rather than round);
* the gradient of an activation function is evaluated in float32: some ulp (2^-20) of its terms' magnitudes.
"""

import numpy as np
import pytest

import oracle.linear8 as ol
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 1e-37, "fp16": 2.0 ** -24, "fp32": 1e-37}       # the smallest step of an output


def _type(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _f64(t):
    return t.detach().double().cpu().numpy()


def _codes(t):
    import torch
    return t.contiguous().view(torch.uint8).cpu().numpy()


def _values(rows, dim, seed, spread=1.0):
    """Unit-scale values with rows and columns of unlike size, zeros among them."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, dim)) * np.exp(spread * rng.standard_normal(dim)) * np.exp(0.5 * rng.standard_normal((rows, 1)))
    x[rng.random((rows, dim)) < 0.05] = 0.0
    return x.astype(np.float32)


def _same_codes(q, want, label):
    codes, byte = (_codes(t) for t in q.unpadded())
    assert np.array_equal(byte, want[1]), f"{label}: scales"
    nan = (want[0] & 0x7F) == 0x7F
    assert np.array_equal(np.where(nan, 0x7F, want[0]), np.where(nan, codes & 0x7F, codes)), f"{label}: codes"
    dim = q.dim
    assert not _codes(q.codes)[:, dim:].any(), f"{label}: padding"


def _weight(w):
    import muon_optimizer_step_amd as ms
    return ms.weight8_encode(w.cuda())


# rows, dim: every width of a unit, ends inside a chunk of 8 and a block, more than one pass
SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 8), (17, 16), (4, 127), (9, 128), (63, 129), (64, 257), (65, 1000), (130, 600),
          (33, 2176), (700, 40)]


@pytest.mark.parametrize("rows,dim", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_encode_to_the_bit(rows, dim, dtype):
    import torch
    import muon_optimizer_step_amd as ms
    gu.say(f"[encode] {rows} x {dim} {dtype}")
    x = torch.from_numpy(_values(rows, dim, rows + dim)).to(_type(dtype))
    want = ol.encode(_f64(x))
    r = ms.act8_encode(x.cuda())
    assert r.out is None
    _same_codes(r.checkpoint, want, "x")
    r = ms.act8_encode(x.cuda(), activation="relu2")
    _same_codes(r.checkpoint, want, "x")
    u = x.float().numpy()
    y = np.where(u > 0, u * u, 0).astype(np.float32)
    _same_codes(r.out, ol.encode(y), "relu2")
    only = ms.act8_encode(x.cuda(), activation="relu2", checkpoint=False)
    assert only.checkpoint is None
    _same_codes(only.out, ol.encode(y), "relu2 alone")


def test_every_bf16_value():
    """All 65536 patterns, NaN and infinities among them, alone in blocks of otherwise smaller or zero values."""
    import torch
    import muon_optimizer_step_amd as ms
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros(65536, 130, dtype=torch.bfloat16)
    x[:, 0], x[:, 5], x[:, 129] = bits, torch.where(torch.isfinite(bits), bits / 3, 1.0), bits
    r = ms.act8_encode(x.cuda())
    got, byte = (_codes(t) for t in r.checkpoint.unpadded())
    want = ol.encode(_f64(x)[:, :130])
    assert np.array_equal(byte, want[1])
    nan = (want[0] & 0x7F) == 0x7F
    assert np.array_equal(nan, (got & 0x7F) == 0x7F)
    assert np.array_equal(got[~nan], want[0][~nan])


def test_rounding_at_every_border():
    """Values at, just below and just above the middle between neighbouring codes, with a fixed scale."""
    import torch
    import muon_optimizer_step_amd as ms
    table = ol.code_values().astype(np.float64)[:127]
    mid = (table[1:] + table[:-1]) / 2
    near = np.concatenate([table, mid, np.nextafter(mid.astype(np.float32), 0), np.nextafter(mid.astype(np.float32), 1e9)])
    near = np.concatenate([near, -near])
    x = np.zeros((len(near), 128), dtype=np.float32)
    x[:, 3], x[:, 77] = near, 448.0
    for power in (-60, 0, 60):
        y = np.ldexp(x, power)
        _same_codes(ms.act8_encode(torch.from_numpy(y).cuda()).checkpoint, ol.encode(y), f"2^{power}")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("rows,dim,dtype", [(1, 40, "bf16"), (65, 300, "fp16"), (130, 1024, "fp32")])
def test_encode_after_smooth_functions(kind, rows, dim, dtype):
    import torch
    import muon_optimizer_step_amd as ms
    x = torch.from_numpy(2 * _values(rows, dim, 7)).to(_type(dtype))
    want = ol.act(_f64(x), kind)
    r = ms.act8_encode(x.cuda(), activation=kind)
    _same_codes(r.checkpoint, ol.encode(_f64(x)), "x")
    codes, byte = (_codes(t) for t in r.out.unpadded())
    assert (np.abs(byte.astype(int) - ol.scales(want)) <= 1).all()
    got = ol.decode(codes, byte)
    scale = np.repeat(2.0 ** (byte.astype(np.float64) - 127), 128, axis=1)[:, :dim]
    tol = (2.0 ** -4 + 2.0 ** -18) * np.abs(want) + (2.0 ** -10 + 2.0 ** -18) * scale
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("kind", ["strided", "unaligned", "odd strides"])
def test_encode_strides_and_alignment(kind):
    import torch
    import muon_optimizer_step_amd as ms
    rows, dim = 70, 200
    pitch, off = {"strided": (256, 0), "unaligned": (dim, 1), "odd strides": (213, 3)}[kind]
    for dtype in ("bf16", "fp32"):
        x = torch.from_numpy(_values(rows, dim, 3)).to(_type(dtype))
        flat = torch.full((rows * pitch + off + 8,), float("nan"), dtype=x.dtype, device="cuda")
        view = flat[off:off + rows * pitch].view(rows, pitch)[:, :dim]
        view.copy_(x)
        _same_codes(ms.act8_encode(view).checkpoint, ol.encode(_f64(x)), kind)
        w8 = ms.weight8_encode(view)
        want = ol.encode(_f64(x), 128)
        _same_codes(w8, want, kind)
        _same_codes(w8.T, (want[0].T, want[1].T), kind)


@pytest.mark.parametrize("rows,dim", [(0, 5), (1, 1), (65, 300), (200, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_decode(rows, dim, dtype):
    import torch
    import muon_optimizer_step_amd as ms
    x = torch.from_numpy(_values(rows, dim, 11))
    q = ms.act8_encode(x.cuda()).checkpoint
    want = torch.from_numpy(ol.decode(*ol.encode(x.numpy()))).to(_type(dtype))
    assert torch.equal(q.decode(_type(dtype)).cpu(), want)
    if rows:
        want = torch.from_numpy(ol.decode(*ol.encode(x.numpy(), 128), 128)).to(_type(dtype))
        w8 = _weight(x)
        assert torch.equal(w8.decode(_type(dtype)).cpu(), want) and torch.equal(w8.T.decode(_type(dtype)).cpu(), want.T)


@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 200), (5, 16), (127, 128), (129, 130), (300, 260), (128, 1030)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_weight_encode(rows, dim, dtype):
    import torch
    import muon_optimizer_step_amd as ms
    gu.say(f"[weight] {rows} x {dim} {dtype}")
    w = torch.from_numpy(_values(rows, dim, rows)).to(_type(dtype))
    if rows > 4 and dim > 4:
        w[1, 2], w[3, 4] = float("nan"), float("-inf")
    want = ol.encode(_f64(w), 128)
    w8 = ms.weight8_encode(w.cuda())
    _same_codes(w8, want, "weight")
    _same_codes(w8.T, (want[0].T, want[1].T), "transposed")
    alone = ms.weight8_encode(w.cuda(), transposed=False)
    _same_codes(alone, want, "alone")
    with pytest.raises(ValueError, match="transpose"):
        alone.T


@pytest.mark.parametrize("dim", [1, 6, 127, 198, 255])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_weight_rows_that_end_inside_a_load(dim, dtype):
    """Aligned rows of an odd length, between values that are none of the matrix: NaN would be seen in the codes."""
    import torch
    import muon_optimizer_step_amd as ms
    w = torch.from_numpy(_values(131, dim, dim)).to(_type(dtype))
    room = torch.full((131, 256), float("nan"), dtype=w.dtype, device="cuda")
    room[:, :dim] = w.cuda()
    want = ol.encode(_f64(w), 128)
    w8 = ms.weight8_encode(room[:, :dim])
    _same_codes(w8, want, "weight")
    _same_codes(w8.T, (want[0].T, want[1].T), "transposed")


@pytest.mark.parametrize("kind", ["relu2", "silu", "gelu"])
@pytest.mark.parametrize("rows,dim,dtype", [(1, 1, "bf16"), (3, 130, "fp16"), (65, 1000, "bf16"), (129, 600, "fp32"), (64, 2048, "fp16")])
def test_backward(kind, rows, dim, dtype):
    import torch
    import muon_optimizer_step_amd as ms
    gu.say(f"[backward] {kind} {rows} x {dim} {dtype}")
    u8 = ms.act8_encode(torch.from_numpy(2 * _values(rows, dim, 5)).cuda()).checkpoint
    grad = torch.from_numpy(_values(rows, dim, 6)).to(_type(dtype))
    u = _f64(u8.decode(torch.float32))
    s, terms = ol.slope(u, kind)
    want = _f64(grad) * s
    r = ms.act8_backward(u8, grad.cuda(), kind, codes=True)
    tol = U[dtype] * np.abs(want) + 2.0 ** -20 * np.abs(_f64(grad)) * terms + TINY[dtype]
    assert (np.abs(_f64(r.grad) - want) <= tol).all()
    if kind == "relu2":
        g32 = (2 * np.maximum(u, 0)).astype(np.float32) * grad.float().numpy()
        _same_codes(r.grad8, ol.encode(g32), "grad8")
    codes, byte = (_codes(t) for t in r.grad8.unpadded())
    scale = np.repeat(2.0 ** (byte.astype(np.float64) - 127), 128, axis=1)[:, :dim]
    tol = (2.0 ** -4 + 2.0 ** -18) * np.abs(want) + 2.0 ** -20 * np.abs(_f64(grad)) * terms + (2.0 ** -10 + 2.0 ** -18) * scale
    assert (np.abs(ol.decode(codes, byte) - want) <= tol).all()
    # in place, and in 8 bits alone
    g = grad.cuda()
    same = ms.act8_backward(u8, g, kind, out=g)
    assert same.grad is g and same.grad8 is None and torch.equal(g, r.grad)
    only = ms.act8_backward(u8, grad.cuda(), kind, out=False, codes=True)
    assert only.grad is None
    for a, b in zip(only.grad8.unpadded(), r.grad8.unpadded()):
        assert np.array_equal(_codes(a), _codes(b))


@pytest.mark.parametrize("kind", ["relu2", "silu", "gelu"])
def test_activations_over_their_whole_range(kind):
    """Every e4m3 value times 2^-12 .. 2^12, zero, NaN and the far ends among them, against the formulas."""
    import torch
    import muon_optimizer_step_amd as ms
    table = np.concatenate([ol.code_values().astype(np.float64)[:127], -ol.code_values().astype(np.float64)[:127]])
    x = np.zeros((25, 256), dtype=np.float32)
    for i, p in enumerate(range(-12, 13)):
        x[i, :127], x[i, 128:255] = np.ldexp(table[:127], p), np.ldexp(table[127:], p)
        x[i, 127], x[i, 255] = np.ldexp(448.0, p), -np.ldexp(448.0, p)
    u8 = ms.act8_encode(torch.from_numpy(x).cuda()).checkpoint
    u = _f64(u8.decode(torch.float32))
    assert np.array_equal(u, x.astype(np.float64))
    with np.errstate(all="ignore"):
        s, terms = ol.slope(u, kind)
        y = ol.act(u, kind)
    got = _f64(ms.act8_backward(u8, torch.ones(25, 256, device="cuda"), kind).grad)
    assert (np.abs(got - s) <= 2.0 ** -20 * terms + 1e-37).all()
    r = ms.act8_encode(torch.from_numpy(x).cuda(), activation=kind, checkpoint=False).out
    codes, byte = (_codes(t) for t in r.unpadded())
    scale = np.repeat(2.0 ** (byte.astype(np.float64) - 127), 128, axis=1)
    assert (np.abs(byte.astype(int) - ol.scales(y)) <= 1).all()
    assert (np.abs(ol.decode(codes, byte) - y) <= (2.0 ** -4 + 2.0 ** -18) * np.abs(y) + (2.0 ** -10 + 2.0 ** -18) * scale).all()
    nan = torch.full((1, 128), float("nan"), device="cuda")
    bad = ms.act8_encode(nan, activation=kind)
    for q in bad:
        assert ((_codes(q.codes) & 0x7F) == 0x7F).all()
    assert torch.isnan(ms.act8_backward(bad.checkpoint, torch.ones(1, 128, device="cuda"), kind).grad).all()


@pytest.mark.parametrize("kind", ["relu2", "silu", "gelu"])
def test_the_slope_is_the_functions(kind):
    """The oracle's derivative against differences of the oracle's function, in 64 bits."""
    u = np.linspace(-6, 6, 2001) + 1e-3
    h = 1e-5
    assert np.abs(ol.slope(u, kind)[0] - (ol.act(u + h, kind) - ol.act(u - h, kind)) / (2 * h)).max() < 1e-8


# ------------------------------------------------------------- products

def _product(rows, cols, dim, dtype, seed=0, **kw):
    import torch
    import muon_optimizer_step_amd as ms
    a8 = ms.act8_encode(torch.from_numpy(_values(rows, dim, seed + 1)).cuda()).checkpoint
    b8 = _weight(torch.from_numpy(_values(cols, dim, seed + 2, 0.3)))
    y = ms.matmul8(a8, b8, dtype=_type(dtype), **kw)
    a, b = _f64(a8.decode(torch.float32)), _f64(b8.decode(torch.float32))
    return y, a, b


def _check_product(y, a, b, dtype, label):
    want = a @ b.T
    tol = (2.0 ** -10 + (a.shape[1] + 16) * 2.0 ** -23) * (np.abs(a) @ np.abs(b).T) * (1 + U[dtype]) + U[dtype] * np.abs(want) + TINY[dtype]
    err = np.abs(_f64(y) - want)
    assert (err <= tol).all(), f"{label}: worst {np.nanmax(err / tol):.3g} of the tolerance"


# rows, cols, dim: few rows, every tile, ends inside tiles, blocks, stages and chunks of 16, more than 16 stages
PRODUCTS = [(1, 1, 1), (1, 4096, 1024), (2, 33, 15), (15, 100, 128), (16, 257, 2200), (17, 64, 129), (31, 31, 255), (33, 130, 600),
            (64, 300, 16), (65, 8, 2304), (127, 129, 384), (128, 128, 128), (129, 255, 1000), (200, 520, 4500), (257, 513, 272),
            (700, 1100, 640), (2050, 2100, 300), (5000, 300, 200)]


@pytest.mark.parametrize("rows,cols,dim", PRODUCTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_matmul(rows, cols, dim, dtype):
    gu.say(f"[matmul8] {rows} x {cols} x {dim} {dtype}")
    y, a, b = _product(rows, cols, dim, dtype)
    _check_product(y, a, b, dtype, "matmul8")


@pytest.mark.parametrize("rows,cols,dim", [(0, 5, 7), (1, 16, 8192), (40, 16, 16384)])
def test_matmul_no_rows_and_long_k(rows, cols, dim):
    y, a, b = _product(rows, cols, dim, "bf16")
    assert tuple(y.shape) == (rows, cols)
    _check_product(y, a, b, "bf16", "long")


@pytest.mark.parametrize("rows,cols,dim", [(20, 70, 66000), (64, 64, 30001)])
def test_matmul_of_many_parts(rows, cols, dim):
    """K in tens of parts, the last one shorter, whose number is no multiple of what the join takes at a time."""
    y, a, b = _product(rows, cols, dim, "fp16")
    _check_product(y, a, b, "fp16", "parts")


@pytest.mark.parametrize("rows,cols,dim", [(5, 64, 512), (64, 512, 2048), (300, 500, 1000), (2050, 2100, 700)])
def test_matmul_error_in_norm(rows, cols, dim):
    """Against the bound of every value above, the errors of random products mostly cancel: in fp16 the output's rounding
    (2^-12 of a value at most, and less on the average) is the larger part."""
    y, a, b = _product(rows, cols, dim, "fp16")
    assert gu.rel_frob(_f64(y), a @ b.T) <= 2.0 ** -12 + 2.0 ** -14


@pytest.mark.parametrize("rows", [3, 40, 300])
def test_matmul_nan_stays_in_its_row_and_column(rows):
    import torch
    import muon_optimizer_step_amd as ms
    x, w = torch.from_numpy(_values(rows, 300, 1)), torch.from_numpy(_values(140, 300, 2))
    x[1, 7], w[130, 299] = float("inf"), float("nan")
    y = _f64(ms.matmul8(ms.act8_encode(x.cuda()).checkpoint, _weight(w)))
    bad = np.isnan(y)
    assert bad[1].all() and bad[:, 130].all() and bad.sum() == rows + 140 - 1


@pytest.mark.parametrize("rows", [5, 70, 300])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_matmul_into_strided_rows(rows, dtype):
    """A slice of a wider output, off the 16-byte grid, and what lies around it untouched."""
    import torch
    import muon_optimizer_step_amd as ms
    a8 = ms.act8_encode(torch.from_numpy(_values(rows, 150, 1)).cuda()).checkpoint
    b8 = _weight(torch.from_numpy(_values(77, 150, 2)))
    want = ms.matmul8(a8, b8, dtype=_type(dtype))
    for pitch, off in ((96, 0), (101, 3)):
        flat = torch.full((rows * pitch + off + 8,), 7.0, dtype=_type(dtype), device="cuda")
        view = flat[off:off + rows * pitch].view(rows, pitch)[:, :77]
        assert ms.matmul8(a8, b8, out=view) is view
        assert torch.equal(view, want)
        view.fill_(7.0)
        assert (flat == 7.0).all()


@pytest.mark.parametrize("scale,power", [(1, 100), (10, 110), (127, 0), (230, -100), (254, -100)])
def test_matmul_takes_any_scale(scale, power):
    """Scales that no encoding of ordinary values gives: 256 x 2^(scale - 127) x 2^power, exact."""
    import torch
    import muon_optimizer_step_amd as ms
    for rows in (4, 90, 300):
        q = ms.act8_encode(torch.ones(rows, 130, device="cuda")).checkpoint      # the code of 256
        a8 = ms.Activation8(q.codes, torch.full_like(q.scale, scale), 130)
        w = torch.zeros(9, 130)
        w[:, 129] = 2.0 ** power
        assert (_f64(ms.matmul8(a8, _weight(w))) == 256.0 * 2.0 ** (scale - 127 + power)).all()


# ------------------------------------------------------------- the weight's gradient

# rows, cols, dim: both tiles, K in one piece and split, ends inside stages and tiles
GRADS = [(1, 1, 1), (1, 300, 200), (3, 8, 16), (63, 65, 129), (64, 128, 128), (65, 129, 15), (128, 16, 257), (200, 300, 260),
         (1000, 64, 64), (1025, 130, 136), (2048, 512, 512), (5000, 72, 300), (130, 1030, 1100), (300, 2304, 2050)]


def _grad_inputs(rows, cols, dim, seed=0):
    import torch
    import muon_optimizer_step_amd as ms
    x8 = ms.act8_encode(torch.from_numpy(_values(rows, dim, seed + 1)).cuda()).checkpoint
    grad = torch.from_numpy(_values(rows, cols, seed + 2)).bfloat16()
    return x8, grad, _f64(x8.decode(torch.float32))


def _check_grad(got, grad, x, before, label):
    g = _f64(grad)
    want = g.T @ x + before
    tol = (len(x) + 48) * 2.0 ** -23 * (np.abs(g).T @ np.abs(x) + np.abs(before)) + 1e-37
    err = np.abs(_f64(got) - want)
    assert (err <= tol).all(), f"{label}: worst {np.nanmax(err / tol):.3g} of the tolerance"


@pytest.mark.parametrize("rows,cols,dim", GRADS + [(33001, 40, 70), (20000, 136, 30)])
def test_grad_weight(rows, cols, dim):
    import torch
    import muon_optimizer_step_amd as ms
    gu.say(f"[grad_weight] {rows} x {cols} x {dim}")
    x8, grad, x = _grad_inputs(rows, cols, dim)
    got = ms.act8_grad_weight(x8, grad.cuda())
    assert got.dtype == torch.float32 and tuple(got.shape) == (cols, dim)
    _check_grad(got, grad, x, 0.0, "grad_weight")
    before = torch.from_numpy(_values(cols, dim, 9))
    out = before.cuda()
    assert ms.act8_grad_weight(x8, grad.cuda(), out=out, accumulate=True) is out
    _check_grad(out, grad, x, _f64(before), "added")


@pytest.mark.parametrize("rows,cols,dim", [(70, 130, 140), (700, 64, 96)])
def test_grad_weight_strides(rows, cols, dim):
    """A gradient that is a slice, on and off the 16-byte grid, into a slice; nothing around it is touched."""
    import torch
    import muon_optimizer_step_amd as ms
    x8, grad, x = _grad_inputs(rows, cols, dim)
    for pitch, off in ((cols + 24, 0), (cols + 24, 8), (cols + 5, 0), (cols, 3)):
        flat = torch.full((rows * pitch + off + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
        view = flat[off:off + rows * pitch].view(rows, pitch)[:, :cols]
        view.copy_(grad)
        wide = torch.full((cols, dim + pitch % 8 + 3), 5.0, device="cuda")
        out = wide[:, pitch % 8:pitch % 8 + dim]
        ms.act8_grad_weight(x8, view, out=out)
        _check_grad(out, grad, x, 0.0, f"{pitch} {off}")
        out.fill_(5.0)
        assert (wide == 5.0).all()


@pytest.mark.parametrize("cols,dim", [(5, 7), (300, 200)])
def test_grad_weight_of_no_rows(cols, dim):
    import torch
    import muon_optimizer_step_amd as ms
    x8 = ms.Activation8.empty(0, dim)
    grad = torch.empty(0, cols, dtype=torch.bfloat16, device="cuda")
    out = torch.full((cols, dim), 3.0, device="cuda")
    assert (ms.act8_grad_weight(x8, grad, out=out, accumulate=True) == 3.0).all()
    assert (ms.act8_grad_weight(x8, grad, out=out) == 0.0).all()


@pytest.mark.parametrize("rows", [10, 64, 100, 1000])
def test_grad_weight_infinities_stay_where_they_belong(rows):
    """An infinite gradient in the last row meets that row's values only: what lies behind the rows is zero."""
    import torch
    import muon_optimizer_step_amd as ms
    x = torch.ones(rows, 40)
    grad = torch.ones(rows, 24)
    grad[-1, 5] = float("inf")
    x[-1, 7] = -1.0
    got = _f64(ms.act8_grad_weight(ms.act8_encode(x.cuda()).checkpoint, grad.bfloat16().cuda()))
    want = (grad.T @ x).double().numpy()
    assert np.array_equal(got, want)
