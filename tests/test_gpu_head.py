"""GPU: the language-model head's loss and gradients against the float64 oracle.

Tolerances, from the arithmetic:
* a logit is a sum of exact products in float32: off by at most (dim + 16) 2^-24 of the sum of magnitudes
  (S below), and a cap adds a few ulp of itself; the log-sum-exp is off by at most as much plus a few ulp of its own
  value and of the base-2 exponents (2^-20 of 1 + |lse|); nll is a difference of two such values;
* P is rounded once to 16 bits, to nearest: by at most u = 2^-8 of itself in bf16 (8 significant bits) and 2^-11 in
  fp16 (11), and its exponentials were kept in fp16, 2^-11 more; so a gradient is off by that share of |P| |W| (or
  |P|^T |H|), and by u of itself for its own rounding.
"""

import numpy as np
import pytest

import oracle.head as oh
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}       # relative error of one rounding
TINY = {"bf16": 1e-30, "fp16": 2.0 ** -24}        # and the smallest step of an output


def _inputs(n, v, d, dtype, seed=0, ignored=0.2):
    import torch
    g = torch.Generator().manual_seed(seed)
    t16 = torch.bfloat16 if dtype == "bf16" else torch.float16
    w = (torch.randn(v, d, generator=g) * (2.5 / d ** 0.5)).to(t16)
    t = torch.randint(0, v, (n,), generator=g)
    h = (torch.randn(n, d, generator=g) + 0.5 * w[t].float()).to(t16)
    t[torch.rand(n, generator=g) < ignored] = -100
    return h, w, t


def _f64(x):
    return x.double().numpy()


def _check(r, want, dim, dtype, cap, grads, label, target=None):
    lim = (dim + 16) * 2.0 ** -24 * want["abs_logit"] + 8 * 2.0 ** -23 * cap
    lse_tol = lim + 2.0 ** -20 * (1 + np.abs(want["lse"]))
    for k, tol in (("lse", lse_tol), ("nll", 2 * lse_tol)):
        err = np.abs(gu.host(getattr(r, k)) - want[k])
        assert (err <= tol).all(), f"{label} {k}: {err.max():.3g} > {tol.min():.3g}"
    if not grads:
        return
    tol = float((2 * lse_tol).max()) + 2.0 ** -20 * abs(want["loss"])
    assert abs(float(r.loss) - want["loss"]) <= tol * max(1.0, grads), f"{label} loss {float(r.loss)} {want['loss']}"
    share = 1.1 * U[dtype] + 2.0 ** -11 + 4 * lim       # P's rounding, e's, and the logits'
    for k, mag in (("grad_hidden", "abs_hidden"), ("grad_weight", "abs_weight")):
        got = getattr(r, k)
        if got is None:
            continue
        got = got.double().cpu().numpy()
        tol = share * want[mag] + 1.01 * U[dtype] * np.abs(want[k]) + TINY[dtype]
        if target is not None:
            tol += target[k](2 * lse_tol)
        err = np.abs(got - want[k])
        assert (err <= tol).all(), f"{label} {k}: worst {np.max(err / tol):.3g} of the tolerance"


# (tokens, vocab, dim): every kernel of the logits, and sizes around its tiles
SMALL = [(1, 1, 1), (1, 5, 8), (3, 64, 7), (31, 65, 64), (32, 127, 72), (33, 129, 100), (64, 128, 63), (65, 130, 129),
         (127, 256, 64), (129, 257, 192), (255, 300, 40), (300, 1000, 130)]
LARGE = [(20, 16400, 72), (50, 16385, 200), (64, 32768, 64), (200, 16500, 65), (1900, 8300, 80), (2048, 8192, 64),
         (2050, 8450, 136)]


@pytest.mark.parametrize("n,v,d", SMALL + LARGE)
@pytest.mark.parametrize("dtype,cap", [("bf16", 0.0), ("fp16", 5.0)])
def test_scores_and_gradients(n, v, d, dtype, cap):
    import muon_optimizer_step_amd as ms
    h, w, t = _inputs(n, v, d, dtype, seed=n + v)
    gu.say(f"[head] {n} x {v} x {d} {dtype} cap {cap}")
    want = oh.head_loss(_f64(h), _f64(w), t.numpy(), softcap=cap)
    hd, wd, td = h.cuda(), w.cuda(), t.cuda()
    _check(ms.linear_cross_entropy(hd, wd, td, softcap=cap), want, d, dtype, cap, 0, "score")
    _check(ms.linear_cross_entropy_grad(hd, wd, td, softcap=cap), want, d, dtype, cap, 1.0, "train")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,v,d", [(5, 40, 24), (70, 600, 64), (400, 3000, 96)])
def test_token_weights(n, v, d, dtype):
    """Weights over six orders of magnitude, negative and zero ones among them."""
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = _inputs(n, v, d, dtype, seed=1)
    rng = np.random.default_rng(n)
    g = (10.0 ** rng.uniform(-4, 2, n) * rng.choice([-1, 0, 1, 1], n) / n).astype(np.float32)
    want = oh.head_loss(_f64(h), _f64(w), t.numpy(), weights=g)
    r = ms.linear_cross_entropy_grad(h.cuda(), w.cuda(), t.cuda(), token_weights=torch.from_numpy(g).cuda())
    _check(r, want, d, dtype, 0.0, float(np.abs(g).sum()), "weighted")


@pytest.mark.parametrize("n", [9, 70, 600])
def test_ignored_tokens_may_hold_anything(n):
    """NaN and infinity in ignored rows reach neither the other tokens nor the gradients."""
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = _inputs(n, 700, 64, "bf16", seed=2, ignored=0.5)
    t[0], t[1] = -100, 3
    bad = h.clone()
    bad[t == -100] = float("nan")
    bad[0] = float("inf")
    want = oh.head_loss(_f64(h), _f64(w), t.numpy())
    r = ms.linear_cross_entropy_grad(bad.cuda(), w.cuda(), t.cuda())
    _check(r, want, 64, "bf16", 0.0, 1.0, "masked")
    gone = (t == -100).numpy()
    assert not gu.host(r.nll)[gone].any() and not gu.host(r.lse)[gone].any()
    assert not r.grad_hidden.float().cpu().numpy()[gone].any()
    s = ms.linear_cross_entropy(bad.cuda(), w.cuda(), t.cuda())
    assert torch.equal(s.nll, r.nll) and torch.equal(s.lse, r.lse)


@pytest.mark.parametrize("n", [0, 1, 40, 300])
def test_no_counted_token(n):
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = _inputs(n, 513, 72, "bf16", seed=3)
    t[:] = 7
    kw = dict(ignore_index=7)
    r = ms.linear_cross_entropy_grad(h.cuda(), w.cuda(), t.cuda(), **kw)
    assert float(r.loss) == 0.0 and torch.count_nonzero(r.grad_weight) == 0 and torch.count_nonzero(r.grad_hidden) == 0
    assert r.nll.shape == (n,) and torch.count_nonzero(r.nll) == 0 and torch.count_nonzero(r.lse) == 0


@pytest.mark.parametrize("target", [-1, 500, 1 << 40, -(1 << 40)])
def test_a_target_outside_the_vocabulary_gives_nan(target):
    import muon_optimizer_step_amd as ms
    h, w, t = _inputs(40, 500, 64, "bf16", seed=4, ignored=0.0)
    t[17] = target
    r = ms.linear_cross_entropy_grad(h.cuda(), w.cuda(), t.cuda())
    nll = gu.host(r.nll)
    assert np.isnan(nll[17]) and np.isfinite(np.delete(nll, 17)).all() and np.isnan(float(r.loss))
    gh = r.grad_hidden.float().cpu().numpy()
    assert np.isnan(gh[17]).all() and np.isfinite(np.delete(gh, 17, axis=0)).all()


@pytest.mark.parametrize("n,v", [(40, 300), (300, 3000), (60, 20000)])
def test_capped_target_far_below_the_maximum(n, v):
    """The target's share of the gradient is - weight x the cap's derivative however small its probability is: targets
    up to 56 below another token's logit, near and far from it in the vocabulary."""
    import torch
    import muon_optimizer_step_amd as ms
    d, cap = 256, 30.0
    h, w, t = _inputs(n, v, d, "bf16", seed=13, ignored=0.0)
    other = (t + torch.randint(1, 40, (n,), generator=torch.Generator().manual_seed(14)) * (1 + 11 * (torch.arange(n) % 2))) % v
    unit = lambda i: w[i].float() / w[i].float().square().sum(1, keepdim=True)  # noqa: E731
    down = torch.linspace(0.0, 50.0, n)[:, None]
    h = (40.0 * unit(other) - down * unit(t)).bfloat16()
    want = oh.head_loss(_f64(h), _f64(w), t.numpy(), softcap=cap)
    assert want["nll"].max() > 50
    r = ms.linear_cross_entropy_grad(h.cuda(), w.cuda(), t.cuda(), softcap=cap)

    # The target's entry is a difference, softmax - 1: an error x of the exponent (of the logit and the log-sum-exp) is
    # x of the softmax, at most x itself, also where the difference is far smaller.
    def in_weight(x):
        out = np.zeros((v, d))
        np.add.at(out, t.numpy(), (x / n)[:, None] * np.abs(_f64(h)))
        return out
    target = {"grad_hidden": lambda x: (x / n)[:, None] * np.abs(_f64(w))[t.numpy()], "grad_weight": in_weight}
    _check(r, want, d, "bf16", cap, 1.0, "far target", target)


def test_infinite_and_huge_logits():
    """Logits of +-1e4 saturate the softmax without overflow; an infinite logit gives NaN in its own row only."""
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = _inputs(70, 300, 64, "bf16", seed=5, ignored=0.0)
    h *= 400.0
    want = oh.head_loss(_f64(h), _f64(w), t.numpy())
    assert want["lse"].max() > 1000
    r = ms.linear_cross_entropy_grad(h.cuda(), w.cuda(), t.cuda())
    _check(r, want, 64, "bf16", 0.0, 1.0, "huge")
    h[5, 3] = float("inf")
    s = ms.linear_cross_entropy(h.cuda(), w.cuda(), t.cuda())
    bad = ~torch.isfinite(s.nll).cpu().numpy()
    assert bad[5] and bad.sum() == 1


@pytest.mark.parametrize("kind", ["strided", "unaligned", "odd strides"])
@pytest.mark.parametrize("n", [20, 300])
def test_strides_and_alignment(kind, n):
    import torch
    import muon_optimizer_step_amd as ms
    v, d = 700, 72
    h, w, t = _inputs(n, v, d, "bf16", seed=6)
    pitch, off = {"strided": (128, 0), "unaligned": (d, 1), "odd strides": (77, 3)}[kind]

    def lay(x):
        flat = torch.full((x.shape[0] * pitch + off + 8,), float("nan"), dtype=x.dtype, device="cuda")
        view = flat[off:off + x.shape[0] * pitch].view(x.shape[0], pitch)[:, :d]
        view.copy_(x)
        return flat, view

    (_, hv), (_, wv) = lay(h), lay(w)
    (gh_flat, gh), (gw_flat, gw) = lay(torch.zeros_like(h)), lay(torch.zeros_like(w))
    want = oh.head_loss(_f64(h), _f64(w), t.numpy())
    r = ms.linear_cross_entropy_grad(hv, wv, t.cuda(), grad_hidden=gh, grad_weight=gw)
    _check(r, want, d, "bf16", 0.0, 1.0, kind)
    for flat, view in ((gh_flat, gh), (gw_flat, gw)):     # nothing between the rows was written
        total, inside = int(torch.isnan(flat).sum()), view.numel()
        assert total == flat.numel() - inside


@pytest.mark.parametrize("which", ["grad_hidden", "grad_weight", "neither"])
def test_one_gradient_alone(which):
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = _inputs(300, 2000, 64, "bf16", seed=7)
    hd, wd, td = h.cuda(), w.cuda(), t.cuda()
    both = ms.linear_cross_entropy_grad(hd, wd, td)
    kw = {k: False for k in ("grad_hidden", "grad_weight") if k != which}
    r = ms.linear_cross_entropy_grad(hd, wd, td, **kw)
    for k in ("grad_hidden", "grad_weight"):
        assert (getattr(r, k) is None) == (k != which)
    # the splits of K may differ: equal to rounding
    if which != "neither":
        a, b = getattr(r, which).double(), getattr(both, which).double()
        assert float((a - b).norm()) <= 4e-3 * float(b.norm())
    assert torch.equal(r.nll, both.nll)
    assert abs(float(r.loss) - float(both.loss)) <= 1e-6 * float(both.loss)


def test_pieces_of_the_tokens_are_one_sum():
    """A vocabulary so large that the tokens take three pieces, against torch in float64."""
    import torch
    import muon_optimizer_step_amd as ms
    v, d = 1 << 20, 16
    n = 2 * ms._lib.MUON_HEAD_PIECE_BYTES // (2 * v) + 188
    h, w, t = (x.cuda() for x in _inputs(n, v, d, "bf16", seed=8, ignored=0.1))
    gu.say(f"[head] pieces {n} x {v} x {d}")
    r = ms.linear_cross_entropy_grad(h, w, t)
    counted = t >= 0
    hf, wf = h.double() * counted[:, None], w.double()
    dw = torch.zeros(v, d, dtype=torch.float64, device="cuda")
    adw = torch.zeros_like(dw)
    for a in range(0, n, 100):
        s = slice(a, a + 100)
        z = torch.mm(hf[s], wf.t().contiguous())
        lse = torch.logsumexp(z, 1)
        idx = torch.arange(z.shape[0], device="cuda")
        nll = (lse - z[idx, t[s].clamp_min(0)]) * counted[s]
        assert float((r.nll[s] - nll).abs().max()) <= 2.0 ** -18 * float(lse.abs().max())
        p = torch.exp(z - lse[:, None])
        p[idx, t[s].clamp_min(0)] -= 1
        p *= counted[s, None] / counted.sum()
        dh = torch.mm(p, wf)
        tol = 2.0 ** -7 * torch.mm(p.abs(), wf.abs()) + 2.0 ** -8 * dh.abs() + 1e-30
        assert bool(((r.grad_hidden[s].double() - dh).abs() <= tol).all())
        pt = p.t().contiguous()
        dw += torch.mm(pt, hf[s])
        adw += torch.mm(pt.abs(), hf[s].abs())
    assert bool(((r.grad_weight.double() - dw).abs() <= 2.0 ** -7 * adw + 2.0 ** -8 * dw.abs() + 1e-30).all())


def test_offsets_beyond_32_bits():
    """A vocabulary matrix of more than 4 GiB: the last rows' logits are those of the last rows."""
    import torch
    import muon_optimizer_step_amd as ms
    n, v, d = 5, 1100000, 2048
    assert v * d * 2 > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(9)
    w = torch.empty(v, d, dtype=torch.bfloat16, device="cuda")
    for a in range(0, v, 100000):
        w[a:a + 100000] = torch.randn(100000, d, generator=g, device="cuda") * (2.0 / d ** 0.5)
    t = torch.tensor([v - 1, 0, v // 2, v - 2, -100], device="cuda")
    h = (torch.randn(n, d, generator=g, device="cuda") + 0.5 * w[t.clamp_min(0)].float()).bfloat16()
    r = ms.linear_cross_entropy(h, w, t)
    z = torch.cat([torch.mm(h.double(), w[a:a + 100000].double().t().contiguous()) for a in range(0, v, 100000)], 1)
    lse = torch.logsumexp(z, 1)
    nll = lse - z[torch.arange(n, device="cuda"), t.clamp_min(0)]
    assert float((r.lse - lse)[:4].abs().max()) <= 1e-4 and float((r.nll - nll)[:4].abs().max()) <= 2e-4
    assert float(r.nll[4]) == 0.0


@pytest.mark.parametrize("n,v,d", [(33, 500, 64), (700, 9000, 128)])
def test_same_bits_every_time_on_any_stream_and_workspace(n, v, d):
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = (x.cuda() for x in _inputs(n, v, d, "bf16", seed=10))
    call = ms.PreparedLinearCrossEntropy(h, w, t, grads=True)
    keep = lambda r: [x.clone() for x in r]  # noqa: E731
    first = keep(call())
    call.workspace.fill_(0xFF)                      # NaN everywhere: contents on entry do not matter
    second = keep(call())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    third = ms.linear_cross_entropy_grad(h, w, t, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("n,v,d", [(1, 300, 64), (20, 17000, 600), (64, 33000, 512), (300, 2000, 64), (300, 20000, 1040),
                                   (2050, 8450, 136), (1100, 40000, 64)])
@pytest.mark.parametrize("cap", [0.0, 12.0])
def test_scores_have_the_bits_of_the_gradients_call(n, v, d, cap):
    """Sums over a token are taken in one order whatever the launch: few and many tokens, few and many partials."""
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = (x.cuda() for x in _inputs(n, v, d, "bf16", seed=15))
    s, r = ms.linear_cross_entropy(h, w, t, softcap=cap), ms.linear_cross_entropy_grad(h, w, t, softcap=cap)
    only = ms.linear_cross_entropy_grad(h, w, t, softcap=cap, grad_hidden=False, grad_weight=False)
    assert torch.equal(s.nll, r.nll) and torch.equal(s.lse, r.lse) and torch.equal(s.nll, only.nll)


@pytest.mark.parametrize("n,v,d", [(20, 900, 64), (300, 3000, 100)])
def test_captured_in_a_graph(n, v, d):
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = (x.cuda() for x in _inputs(n, v, d, "bf16", seed=11))
    a = ms.PreparedLinearCrossEntropy(h, w, t, grads=True)
    b = ms.PreparedLinearCrossEntropy(h, w, t, grads=True)
    a()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        a()
    for k in range(4):
        h.copy_(torch.randn(n, d, device="cuda"))
        for x in a.result:
            x.fill_(float("nan"))
        g.replay()
        b()
        float(torch.randn(1 << 16, device="cuda").sum())
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.result, b.result)), k


def test_gradient_against_differences_of_the_loss():
    """The loss's own central difference along a direction, at steps that are exact in fp16."""
    import torch
    import muon_optimizer_step_amd as ms
    n, v, d = 64, 300, 32
    rng = np.random.default_rng(12)
    grid = lambda *s: torch.from_numpy(rng.integers(-64, 65, s) / 64.0)  # noqa: E731
    h, w = grid(n, d), grid(v, d) / 2
    t = torch.from_numpy(rng.integers(0, v, n)).cuda()
    loss = lambda h, w: float(ms.linear_cross_entropy_grad(h.half().cuda(), w.half().cuda(), t).loss)  # noqa: E731
    r = ms.linear_cross_entropy_grad(h.half().cuda(), w.half().cuda(), t)
    for x, grad, which in ((h, r.grad_hidden, 0), (w, r.grad_weight, 1)):
        u = torch.from_numpy(rng.choice([-1.0, 1.0], tuple(x.shape))) / 64      # x +- u is exact
        up, down = (loss(*((x + s * u, w) if which == 0 else (h, x + s * u))) for s in (1, -1))
        want = float((grad.double().cpu() * u).sum())
        # third-order term: |u|_1 rows of 32/64 move logits by <= 0.5, relative error <= 0.5^2; fp32 loss: 1e-6
        assert abs((up - down) / 2 - want) <= 0.1 * abs(want) + 2e-4, (up, down, want)


def test_binding_refusals():
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = (x.cuda() for x in _inputs(8, 100, 64, "bf16"))
    for bad in (dict(targets=t.int()), dict(hidden=h.half()), dict(hidden=h.float()), dict(token_weights=t)):
        kw = dict(hidden=h, weight=w, targets=t, token_weights=None)
        kw.update(bad)
        with pytest.raises(TypeError):
            ms.linear_cross_entropy_grad(kw["hidden"], kw["weight"], kw["targets"], token_weights=kw["token_weights"])
    for a, b, c in ((h[:, :32], w, t), (h, w, t[:4]), (h.t(), w, t), (h, w.cpu(), t), (h[0], w, t)):
        with pytest.raises((ValueError, TypeError)):
            ms.linear_cross_entropy(a, b, c)
    with pytest.raises(ValueError, match="grads=True"):
        ms.PreparedLinearCrossEntropy(h, w, t, token_weights=torch.ones(8, device="cuda"))
    with pytest.raises(ValueError, match="rows overlap"):
        ms.linear_cross_entropy(h[0].expand(8, 64), w, t)
    with pytest.raises(ms.MuonError) as e:
        ms.linear_cross_entropy(h, w, t, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == ms._lib.MUON_ERR_WORKSPACE
    with pytest.raises(ms.MuonError):
        ms.linear_cross_entropy(h, w, t, softcap=-1.0)
