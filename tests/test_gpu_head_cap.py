"""GPU: the head's loss under caps far from the size of the logits, on either side.

A capped logit is cap tanh(z / cap) to a few ulp of itself, whatever the cap: its error stays within that of z, so the
tolerances are those of the uncapped loss (test_gpu_head.py with a cap of 0).
"""

import numpy as np
import pytest

import oracle.head as oh
from tests import gpu_util as gu
from tests.test_gpu_head import _check, _f64, _inputs

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
