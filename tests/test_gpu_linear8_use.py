"""GPU: the linear layers in 8 bits as a program uses them: a layer's whole forward and backward pass, streams, captured
graphs, dropped and reused tensors, buffers past 32 bits, refusals of the binding."""

import gc
import importlib.util
import math
import os
import weakref

import numpy as np
import pytest

import oracle.linear8 as ol
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _f64(t):
    return t.detach().double().cpu().numpy()


def _mlp_inputs(n, d, h, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return (randn(n, d).bfloat16().cuda(), (randn(h, d) / d ** 0.5).cuda(), (randn(d, h) / h ** 0.5).cuda(),
            (1e-2 * randn(n, d)).bfloat16().cuda())


def _mlp(x, w1, w2, dy, act):
    """Every call of a layer x -> act(x w1^T) w2^T and back; returns all that it makes."""
    import muon_optimizer_step_amd as ms
    w18, w28 = ms.weight8_encode(w1), ms.weight8_encode(w2)
    x8 = ms.act8_encode(x).checkpoint
    u = ms.matmul8(x8, w18)
    kept = ms.act8_encode(u, activation=act)
    y = ms.matmul8(kept.out, w28)
    dh = ms.matmul8(ms.act8_encode(dy).checkpoint, w28.T)
    back = ms.act8_backward(kept.checkpoint, dh, act, codes=True)
    dw2 = ms.act8_grad_weight(kept.out, dy)
    dw1 = ms.act8_grad_weight(x8, back.grad)
    dx = ms.matmul8(back.grad8, w18.T)
    return dict(w18=w18, w28=w28, x8=x8, u=u, u8=kept.checkpoint, h8=kept.out, y=y, dh=dh, du=back.grad, du8=back.grad8, dw1=dw1,
                dw2=dw2, dx=dx)


def _tensors(r):
    out = {}
    for k, v in r.items():
        if hasattr(v, "unpadded"):
            out[k + ".codes"], out[k + ".scale"] = (t.contiguous().view(__import__("torch").uint8) for t in v.unpadded())
        else:
            out[k] = v
    return out


@pytest.mark.parametrize("act", ["relu2", "silu", "gelu"])
@pytest.mark.parametrize("n,d,h", [(1, 64, 256), (70, 100, 333), (600, 512, 2048)])
def test_a_layer_forward_and_back(act, n, d, h):
    """Each step against 64 bits from what the step before it gave, and the whole against the exact layer, to the 8-bit
    roundings (2^-4 of a value each, uniform: a standard deviation of 2^-4 / 3 or so of it, less where they average)."""
    x, w1, w2, dy = _mlp_inputs(n, d, h)
    gu.say(f"[layer] {act} {n} x {d} x {h}")
    r = _mlp(x, w1, w2, dy, act)
    val = {k: _f64(r[k].decode()) for k in ("w18", "w28", "x8", "u8", "h8", "du8")}
    rel = lambda got, want: np.linalg.norm(_f64(got) - want) / np.linalg.norm(want)  # noqa: E731
    assert rel(r["u"], val["x8"] @ val["w18"].T) < 2.0 ** -8
    assert rel(r["y"], val["h8"] @ val["w28"].T) < 2.0 ** -8
    s, _ = ol.slope(val["u8"], act)
    assert rel(r["du"], _f64(r["dh"]) * s) < 2.0 ** -8
    assert rel(r["dw2"], _f64(dy).T @ val["h8"]) < 1e-5
    assert rel(r["dw1"], _f64(r["du"]).T @ val["x8"]) < 1e-5
    assert rel(r["dx"], val["du8"] @ val["w18"]) < 2.0 ** -8
    X, W1, W2, DY = (_f64(t) for t in (x, w1, w2, dy))
    u = X @ W1.T
    slope, _ = ol.slope(u, act)
    du = (DY @ W2) * slope
    whole = {"y": ol.act(u, act) @ W2.T, "dw2": DY.T @ ol.act(u, act), "dw1": du.T @ X, "dx": du @ W1}
    for k, want in whole.items():
        assert rel(r[k], want) < 0.15, k


@pytest.mark.parametrize("act", ["relu2", "silu", "gelu"])
def test_the_gradients_against_differences(act):
    """The backward pass's formulas, followed by the calls above to their roundings, against differences of the layer in
    64 bits."""
    rng = np.random.default_rng(3)
    x, w1, w2, c = (rng.standard_normal(s) for s in ((5, 6), (7, 6), (6, 7), (5, 6)))
    loss = lambda a, b, e: float((ol.act(a @ b.T, act) @ e.T * c).sum())  # noqa: E731
    u = x @ w1.T
    du = (c @ w2) * ol.slope(u, act)[0]
    for i, (t, g) in enumerate(((x, du @ w1), (w1, du.T @ x), (w2, c.T @ ol.act(u, act)))):
        for at in ((0, 0), (3, 2), (t.shape[0] - 1, t.shape[1] - 1)):
            args = [[x, w1, w2], [x, w1, w2]]
            for side, step in ((0, 1e-6), (1, -1e-6)):
                moved = t.copy()
                moved[at] += step
                args[side][i] = moved
            assert abs((loss(*args[0]) - loss(*args[1])) / 2e-6 - g[at]) < 1e-6 * (1 + abs(g[at]))


def test_the_same_bits_every_time():
    import torch
    for n, d, h in ((3, 512, 2048), (200, 300, 1000), (2100, 512, 2048)):
        args = _mlp_inputs(n, d, h)
        first = _tensors(_mlp(*args, "silu"))
        for _ in range(3):
            again = _tensors(_mlp(*args, "silu"))
            assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("n", [1, 40, 700, 3000])
def test_captured_and_replayed(n):
    """All calls in one graph, replayed with new inputs and eager work between the replays."""
    import torch
    x, w1, w2, dy = _mlp_inputs(n, 256, 1024)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _mlp(x, w1, w2, dy, "relu2")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = _tensors(_mlp(x, w1, w2, dy, "relu2"))
    for seed in range(4):
        for t, new in zip((x, w1, w2, dy), _mlp_inputs(n, 256, 1024, seed)):
            t.copy_(new)
        graph.replay()
        got = {k: v.clone() for k, v in r.items()}
        torch.cuda.synchronize()
        want = _tensors(_mlp(x, w1, w2, dy, "relu2"))
        assert all(torch.equal(got[k], want[k]) for k in want), seed


def test_two_graphs_share_nothing():
    import torch
    import muon_optimizer_step_amd as ms
    a8 = ms.act8_encode(torch.randn(64, 8192, device="cuda")).checkpoint        # K split: both have partial sums
    grad = torch.randn(3000, 128, device="cuda").bfloat16()
    x8 = ms.act8_encode(torch.randn(3000, 128, device="cuda")).checkpoint
    ws = [ms.weight8_encode(torch.randn(512, 8192, device="cuda")) for _ in range(2)]
    want = [(ms.matmul8(a8, w), ms.act8_grad_weight(x8, grad * k)) for k, w in enumerate(ws, 1)]
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph() for _ in ws], []
    for k, (g, w) in enumerate(zip(graphs, ws), 1):
        scaled = grad * k
        with torch.cuda.graph(g):
            got.append((ms.matmul8(a8, w), ms.act8_grad_weight(x8, scaled)))
    streams = [torch.cuda.Stream() for _ in ws]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for a, b in zip(got, want) for p, q in zip(a, b))


def test_inputs_dropped_after_a_call_on_another_stream():
    import torch
    import muon_optimizer_step_amd as ms
    x, w1, w2, dy = _mlp_inputs(700, 256, 1024)
    want = _mlp(x, w1, w2, dy, "gelu")
    side = torch.cuda.Stream()

    def late(call, *tensors):
        """call(copies of the tensors) on the busy side stream; the copies' memory is taken over at once."""
        copies = [t.clone() for t in tensors]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000_000)
        out = call(*copies)
        del copies
        junk = [torch.full_like(t, 0 if t.dtype == torch.uint8 else float("nan")) for t in tensors for _ in range(3)]
        torch.cuda.synchronize()
        del junk
        return out

    same = lambda a, b: all(torch.equal(p, q) for p, q in zip(_tensors({"r": a}).values(), _tensors({"r": b}).values()))  # noqa: E731
    coded = lambda q: (q.codes.view(torch.uint8), q.scale)  # noqa: E731
    act = lambda c, s, like: ms.Activation8(c.view(torch.float8_e4m3fn), s, like.dim)  # noqa: E731
    wgt = lambda c, s, like: ms.Weight8(c.view(torch.float8_e4m3fn), s, like.dim)  # noqa: E731
    assert same(late(lambda t: ms.act8_encode(t, stream=side).checkpoint, x), want["x8"])
    assert same(late(lambda t: ms.weight8_encode(t, stream=side).T, w1), want["w18"].T)
    assert same(late(lambda a, b, c, d: ms.matmul8(act(a, b, want["x8"]), wgt(c, d, want["w18"]), stream=side), *coded(want["x8"]),
                     *coded(want["w18"])), want["u"])
    assert same(late(lambda a, b, g: ms.act8_backward(act(a, b, want["u8"]), g, "gelu", stream=side).grad, *coded(want["u8"]),
                     want["dh"]), want["du"])
    assert same(late(lambda a, b, g: ms.act8_grad_weight(act(a, b, want["x8"]), g, stream=side), *coded(want["x8"]), want["du"]),
                want["dw1"])
    assert same(late(lambda a, b: act(a, b, want["x8"]).decode(stream=side), *coded(want["x8"])), want["x8"].decode())


def test_prepared_calls_keep_their_tensors():
    import torch
    import muon_optimizer_step_amd as ms
    x, w, dy = torch.randn(30, 64, device="cuda"), torch.randn(40, 64, device="cuda"), torch.randn(30, 40, device="cuda").bfloat16()
    x8, w8 = ms.act8_encode(x).checkpoint, ms.weight8_encode(w)
    calls = [ms.PreparedAct8Encode(x), ms.PreparedWeight8Encode(w), ms.PreparedMatmul8(x8, w8), ms.PreparedAct8GradWeight(x8, dy),
             ms.PreparedAct8Backward(x8, x, "silu")]
    refs = [weakref.ref(t) for t in (x, w, dy, x8.codes, x8.scale, w8.codes, w8.scale)]
    del x, w, dy, x8, w8
    gc.collect()
    assert all(r() is not None for r in refs)
    first = [c() for c in calls]
    assert all(a is b for a, b in zip(first, [c() for c in calls]))


def test_accumulated_over_microbatches():
    """Gradients of three microbatches added in place give that of the three as one, to the sums' rounding."""
    import torch
    import muon_optimizer_step_amd as ms
    x, dy = torch.randn(900, 136, device="cuda"), torch.randn(900, 72, device="cuda").bfloat16()
    x8 = ms.act8_encode(x).checkpoint
    out = torch.zeros(72, 136, device="cuda")
    for a in (0, 300, 600):
        part = ms.Activation8(x8.codes[a:a + 300], x8.scale[a:a + 300], 136)
        ms.act8_grad_weight(part, dy[a:a + 300], out=out, accumulate=True)
    want = _f64(dy).T @ _f64(x8.decode())
    bound = np.abs(_f64(dy)).T @ np.abs(_f64(x8.decode()))
    assert (np.abs(_f64(out) - want) <= 1000 * 2.0 ** -23 * bound).all()


def test_muon_takes_the_gradient():
    """The float32 gradient goes into PreparedMuonStep as it is, and the updated weight into the next encoding."""
    import torch
    import muon_optimizer_step_amd as ms
    w = torch.randn(256, 128, device="cuda")
    grad, mom = torch.empty_like(w), torch.zeros_like(w)
    encode = ms.PreparedWeight8Encode(w)
    step = ms.PreparedMuonStep([w], [grad], [mom])
    x = torch.randn(500, 128, device="cuda")
    x8 = ms.act8_encode(x).checkpoint
    for _ in range(2):
        w8 = encode()
        y = ms.matmul8(x8, w8)
        ms.act8_grad_weight(x8, y, out=grad)
        step(lr=0.1, momentum=0.9, weight_decay=0.0, coeffs=[(3.4445, -4.7750, 2.0315)] * 5)
    want, byte = ol.encode(_f64(w), 128)
    codes, scale = encode().unpadded()
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), want) and np.array_equal(scale.cpu().numpy(), byte)


def test_past_32_bits():
    """Codes, values and gradients of over 2^32 bytes: the last rows' results are those of the last rows alone."""
    import torch
    import muon_optimizer_step_amd as ms
    rows, dim = 530_000, 8192
    x = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    last = slice(rows - 200, rows)
    x[last] = torch.randn(200, dim, device="cuda").bfloat16()
    r = ms.act8_encode(x, activation="relu2")
    tail = ms.act8_encode(x[last], activation="relu2")
    cut = lambda q: ms.Activation8(q.codes[last], q.scale[last], dim)  # noqa: E731
    eq = lambda p, q: all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(p.unpadded(), q.unpadded()))  # noqa: E731
    assert r.checkpoint.codes.numel() > 1 << 32
    assert eq(cut(r.checkpoint), tail.checkpoint) and eq(cut(r.out), tail.out)
    w8 = ms.weight8_encode(torch.randn(48, dim, device="cuda") / 90)
    y, z = ms.matmul8(r.checkpoint, w8), ms.matmul8(tail.checkpoint, w8)
    assert gu.rel_frob(_f64(y[last]), _f64(z)) < 2.0 ** -8 and not y[:rows - 200].any()
    grad = torch.zeros(rows, 48, dtype=torch.bfloat16, device="cuda")
    grad[last] = torch.randn(200, 48, device="cuda").bfloat16()
    got, want = ms.act8_grad_weight(r.checkpoint, grad), ms.act8_grad_weight(tail.checkpoint, grad[last])
    assert gu.rel_frob(_f64(got), _f64(want)) < 1e-6
    back = ms.act8_backward(r.checkpoint, x, "relu2", out=x)
    u = _f64(tail.checkpoint.decode(torch.float32))
    assert np.isfinite(_f64(back.grad[last])).all() and (_f64(back.grad[last]) != 0).sum() > (u > 0).sum() * 0.9


# ------------------------------------------------------------- refusals

def test_refusals_of_the_binding():
    import torch
    import muon_optimizer_step_amd as ms
    x, w = torch.randn(20, 64, device="cuda"), torch.randn(30, 64, device="cuda")
    x8, w8 = ms.act8_encode(x).checkpoint, ms.weight8_encode(w)
    dy = torch.randn(20, 30, device="cuda").bfloat16()
    for call, error, words in (
            (lambda: ms.act8_encode(x.cpu()), ValueError, "HIP device"),
            (lambda: ms.act8_encode(x.double()), TypeError, "float64"),
            (lambda: ms.act8_encode(x[0]), ValueError, "2-D"),
            (lambda: ms.act8_encode(x.t()), ValueError, "contiguous rows"),
            (lambda: ms.act8_encode(x.as_strided((20, 64), (32, 1))), ValueError, "overlap"),
            (lambda: ms.act8_encode(x, activation="tanh"), ValueError, "activation"),
            (lambda: ms.act8_encode(x, checkpoint=False), ValueError, "nothing to encode"),
            (lambda: ms.act8_encode([1.0]), TypeError, "torch.Tensor"),
            (lambda: ms.weight8_encode(w[:0]), ValueError, "empty"),
            (lambda: ms.weight8_encode(w, transposed=False).T, ValueError, "transpose"),
            (lambda: ms.Activation8(x8.codes, x8.scale, 70), ValueError, "columns"),
            (lambda: ms.Activation8(x8.codes, x8.scale[:5]), ValueError, "scale"),
            (lambda: ms.Activation8(x8.codes.view(torch.uint8), x8.scale), TypeError, "float8"),
            (lambda: ms.Activation8(x8.codes, w8.scale), ValueError, "scale"),
            (lambda: ms.Activation8.empty(3, 0), ValueError, "dim >= 1"),
            (lambda: ms.matmul8(x8, x8), TypeError, "Weight8"),
            (lambda: ms.matmul8(w8, w8), TypeError, "Activation8"),
            (lambda: ms.matmul8(x8, w8.T), ValueError, "columns"),
            (lambda: ms.matmul8(x8, w8, dtype=torch.float32), TypeError, "bfloat16"),
            (lambda: ms.matmul8(x8, w8, out=torch.empty(20, 31, device="cuda", dtype=torch.bfloat16)), ValueError, "shape"),
            (lambda: ms.matmul8(x8, w8, out=torch.empty(20, 30, device="cuda")), TypeError, "out"),
            (lambda: ms.matmul8(x8, w8, workspace=torch.empty(8, device="cuda")), ms.MuonError, "workspace"),
            (lambda: ms.matmul8(x8, w8, workspace=torch.empty(512)), ValueError, "workspace"),
            (lambda: ms.act8_grad_weight(x8, dy.half()), TypeError, "bfloat16"),
            (lambda: ms.act8_grad_weight(x8, dy[:19]), ValueError, "shape"),
            (lambda: ms.act8_grad_weight(x8, dy, accumulate=True), ValueError, "out"),
            (lambda: ms.act8_grad_weight(x8, dy, out=torch.empty(30, 63, device="cuda")), ValueError, "shape"),
            (lambda: ms.act8_backward(x8, x, "none"), ValueError, "none"),
            (lambda: ms.act8_backward(x8, x[:, :60], "relu2"), ValueError, "shape"),
            (lambda: ms.act8_backward(x8, x, "relu2", out=False), ValueError, "nothing to compute"),
            (lambda: ms.act8_backward(x8, x, "relu2", out=x.half()), TypeError, "out"),
            (lambda: x8.decode(torch.float64), TypeError, "dtype"),
    ):
        with pytest.raises(error, match=words):
            call()
    # what is written may not overlap what is read, but for a gradient in place
    wide = torch.randn(20, 128, device="cuda")
    with pytest.raises(ms.MuonError, match="overlap"):
        ms.act8_backward(x8, wide[:, :64], "relu2", out=wide[:, 32:96])
    both = torch.zeros(20 * 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).view(20, 64)
    alias = ms.Activation8(both, x8.scale)
    with pytest.raises(ms.MuonError, match="overlap"):
        ms.matmul8(alias, w8, out=both.view(torch.uint8).view(-1)[:1200].view(torch.bfloat16).view(20, 30))


def test_a_single_row_has_no_row_stride():
    import torch
    import muon_optimizer_step_amd as ms
    x, w = torch.randn(1, 64, device="cuda"), torch.randn(30, 64, device="cuda")
    wide = torch.as_strided(x, (1, 64), (1 << 30, 1))
    a, b = ms.act8_encode(wide).checkpoint, ms.act8_encode(x).checkpoint
    w8 = ms.weight8_encode(w)
    far = ms.Activation8(torch.as_strided(b.codes, (1, 64), (1 << 30, 1)), b.scale)
    assert torch.equal(ms.matmul8(a, w8), ms.matmul8(b, w8)) and torch.equal(ms.matmul8(far, w8), ms.matmul8(b, w8))


# ------------------------------------------------------------- the example

def _example():
    spec = importlib.util.spec_from_file_location("train_lm_head", os.path.join(ROOT, "examples", "train_lm_head.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def test_example_runs_with_linear8():
    losses = _example().train(vocab=512, dim=128, tokens=2048, steps=4, linear8=True)
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses) and abs(losses[0] - math.log(512)) < 1.0


def test_example_layers_gradients():
    """Linear8 against the same layer in 64 bits on the values that its codes stand for."""
    import torch
    import muon_optimizer_step_amd as ms
    ex = _example()
    x, w = torch.randn(300, 128, device="cuda", requires_grad=True), torch.randn(64, 128, device="cuda") / 11
    w8, w_grad = ms.weight8_encode(w), torch.empty_like(w)
    y = ex.Linear8.apply(x, w8, w_grad)
    dy = torch.randn(300, 64, device="cuda").bfloat16()
    dx, = torch.autograd.grad(y, x, dy)
    X, W, D = _f64(ms.act8_encode(x.detach()).checkpoint.decode()), _f64(w8.decode()), _f64(dy)
    D8 = _f64(ms.act8_encode(dy).checkpoint.decode())
    assert gu.rel_frob(_f64(y), X @ W.T) < 2.0 ** -8 and gu.rel_frob(_f64(w_grad), D.T @ X) < 1e-5
    assert gu.rel_frob(_f64(dx), D8 @ W) < 2.0 ** -8
