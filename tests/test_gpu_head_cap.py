"""GPU: the head's loss under caps far from the size of the logits, on either side.

A capped logit is cap tanh(z / cap) to a few ulp of itself, whatever the cap: its error stays within that of z, so the
tolerances are those of the uncapped loss (test_gpu_head.py with a cap of 0).
"""

import numpy as np
import pytest

import oracle.head as oh
from tests import gpu_util as gu
from tests.test_gpu_head import TINY, U, _check, _f64, _inputs

pytestmark = pytest.mark.gpu


# (tokens, vocab, dim): each kernel of the logits
SMALL = [(20, 900, 64), (20, 16400, 72), (50, 900, 72), (300, 3000, 100)]
LARGE = (2050, 8450, 64)
CAPS = [1e-40, 1e-3, 0.5, 3.0, 50.0, 1e3, 1e6, 1e30, 3e38]


@pytest.mark.parametrize("n,v,d,cap", [(*s, c) for s in SMALL for c in CAPS] + [(*LARGE, 3.0), (*LARGE, 1e6)])
def test_capped_logits_keep_their_digits(n, v, d, cap):
    import muon_optimizer_step_amd as ms
    dtype = "bf16" if n % 20 else "fp16"
    h, w, t = _inputs(n, v, d, dtype, seed=n)
    gu.say(f"[head cap] {n} x {v} x {d} {dtype} cap {cap}")
    want = oh.head_loss(_f64(h), _f64(w), t.numpy(), softcap=float(np.float32(cap)))
    _check(ms.linear_cross_entropy(h.cuda(), w.cuda(), t.cuda(), softcap=cap), want, d, dtype, 0.0, 0, f"cap {cap}")
    if cap >= 50.0:
        _check(ms.linear_cross_entropy_grad(h.cuda(), w.cuda(), t.cuda(), softcap=cap), want, d, dtype, 0.0, 1.0, f"cap {cap}")


@pytest.mark.parametrize("n,v,d", [(20, 300, 64), (200, 600, 64)])
def test_a_cap_bounds_infinite_logits(n, v, d):
    """cap tanh of an infinite logit is +-cap: nll and lse stay finite."""
    import torch
    import muon_optimizer_step_amd as ms
    cap = 4.0
    h, w, t = _inputs(n, v, d, "bf16", seed=21, ignored=0.0)
    h[:, 0], w[:, 0] = 1.0, 0.0
    w[7, 0], w[v - 1, 0] = float("inf"), -float("inf")
    z = _f64(h[:, 1:]) @ _f64(w[:, 1:]).T
    z[:, 7], z[:, v - 1] = np.inf, -np.inf
    t[3] = 7
    lo = cap * np.tanh(z / cap)
    lse = np.log(np.exp(lo).sum(1))
    nll = lse - lo[np.arange(n), t.numpy()]
    r = ms.linear_cross_entropy(h.cuda(), w.cuda(), t.cuda(), softcap=cap)
    lim = (d + 16) * 2.0 ** -24 * float((np.abs(_f64(h[:, 1:])) @ np.abs(_f64(w[:, 1:])).T).max()) + 2.0 ** -20 * (1 + lse)
    assert (np.abs(gu.host(r.lse) - lse) <= lim).all() and (np.abs(gu.host(r.nll) - nll) <= 2 * lim).all()


@pytest.mark.parametrize("n,v,d", [(20, 900, 64), (50, 900, 72), (300, 3000, 100), (2050, 8450, 64)])
@pytest.mark.parametrize("cap,lo,hi", [(0.5, 2.0, 6.0), (5.0, 3.0, 5.0), (30.0, 3.0, 7.0), (30.0, 0.2, 3.0)])
def test_gradients_of_saturated_logits(n, v, d, cap, lo, hi):
    """Every logit, not the target's alone, is lo .. hi caps from zero, where the cap's derivative is down to 4 exp(-2 hi).

    Tolerance of an entry of P, on top of test_gpu_head.py's share of it: the derivative's relative error from that of
    z (2 / cap of it) and of its own arithmetic (2^-20 (1 + 2 hi)); and, where the entry is far below the largest of
    its neighbours, an absolute 2^-37 of the token's weight (the smallest steps of fp16: 2^-25 of exponentials that
    reach 2^15, and 2^-25 of probabilities in units of 2^-13).
    """
    import torch
    import muon_optimizer_step_amd as ms
    dtype = "bf16" if n % 20 else "fp16"
    t16 = torch.bfloat16 if dtype == "bf16" else torch.float16
    g = torch.Generator().manual_seed(n + v)
    a = torch.randn(d, generator=g)
    sign = torch.randint(0, 2, (v, 1), generator=g) * 2.0 - 1.0
    w = (sign * a * (1 + 0.02 * torch.randn(v, d, generator=g))).to(t16)
    c = cap * (lo + (hi - lo) * torch.rand(n, 1, generator=g))
    h = (c * a / a.square().sum()).to(t16)
    t = torch.randint(0, v, (n,), generator=g)
    t[1] = -100
    gu.say(f"[head cap] saturated {n} x {v} x {d} {dtype} cap {cap}")
    hf, wf = _f64(h), _f64(w)
    want = oh.head_loss(hf, wf, t.numpy(), softcap=cap)
    lim = (d + 16) * 2.0 ** -24 * want["abs_logit"]
    lse_tol = lim + 2.0 ** -20 * (1 + np.abs(want["lse"]))
    counted = (t >= 0).numpy()
    share = 1.1 * U[dtype] + 2.0 ** -11 + (4 + 2 / cap) * lim + 2.0 ** -20 * (1 + 2 * hi)
    weight = counted / counted.sum()
    # the target's entry is a difference, softmax - 1
    off = weight * (2 * lse_tol + 2.0 ** -11) * (1 - np.tanh((hf * wf[np.where(counted, t.numpy(), 0)]).sum(1) / cap) ** 2)
    in_weight = np.zeros((v, d))
    np.add.at(in_weight, np.where(counted, t.numpy(), 0), off[:, None] * np.abs(hf))
    r = ms.linear_cross_entropy_grad(h.cuda(), w.cuda(), t.cuda(), softcap=cap)
    for k, mag, more in (("grad_hidden", "abs_hidden", off[:, None] * np.abs(wf)[np.where(counted, t.numpy(), 0)]
                          + 2.0 ** -37 * weight[:, None] * np.abs(wf).sum(0)),
                         ("grad_weight", "abs_weight", in_weight + 2.0 ** -37 * (weight[:, None] * np.abs(hf)).sum(0))):
        got = getattr(r, k).double().cpu().numpy()
        tol = share * want[mag] + 1.01 * U[dtype] * np.abs(want[k]) + TINY[dtype] + more
        err = np.abs(got - want[k])
        gu.say(f"  {k}: worst {np.max(err / tol):.3g} of the tolerance, relative {np.linalg.norm(got - want[k]) / np.linalg.norm(want[k]):.3g}")
        assert (err <= tol).all(), f"{k}: worst {np.max(err / tol):.3g} of the tolerance"


@pytest.mark.parametrize("n,v,d", [(20, 900, 64), (300, 3000, 100)])
@pytest.mark.parametrize("cap", [1e-40, 1e-3])
def test_gradients_under_a_tiny_cap(n, v, d, cap):
    """Logits of 0.9 and more, hundreds of caps from zero: the derivative, at most 4 exp(-1800), and the gradients vanish."""
    import torch
    import muon_optimizer_step_amd as ms
    g = torch.Generator().manual_seed(n)
    a = torch.randn(d, generator=g)
    sign = torch.randint(0, 2, (v, 1), generator=g) * 2.0 - 1.0
    h = ((1 + torch.rand(n, 1, generator=g)) * a / a.square().sum()).bfloat16()
    r = ms.linear_cross_entropy_grad(h.cuda(), (sign * a).bfloat16().cuda(), torch.randint(0, v, (n,), generator=g).cuda(),
                                     softcap=cap)
    assert torch.count_nonzero(r.grad_hidden) == 0 and torch.count_nonzero(r.grad_weight) == 0
