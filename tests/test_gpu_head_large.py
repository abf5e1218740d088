"""GPU: the head's loss where a problem takes several pieces, or its exponentials go past the caches.

The oracle is torch in float64 on the GPU, a part of the tokens at a time (products with a contiguous right operand).
Tolerances are test_gpu_head.py's, with what its sizes leave out: a probability far below the largest of its neighbours
(or of the weight, in fp16) is kept to an absolute 2^-37 of the token's weight, the smallest steps of fp16 (2^-25 of
exponentials that reach 2^15, and 2^-25 of probabilities in units of 2^-13); and the cap's derivative is off by 2 / cap
of the logit's error and by its own arithmetic.
"""

import pytest

from tests import gpu_util as gu
from tests.test_gpu_head import TINY, U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,v", [(300, 4194304), (384, 2800000), (330, 3300000)])
def test_scores_have_the_bits_of_a_call_in_pieces(n, v):
    """Sums over a token are taken in one order also where the gradients' call works in pieces and scoring does not."""
    import torch
    import muon_optimizer_step_amd as ms
    g = torch.Generator(device="cuda").manual_seed(n)
    gu.say(f"[head large] bits {n} x {v} x 8")
    h = torch.randn(n, 8, generator=g, device="cuda").bfloat16()
    w = torch.randn(v, 8, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    s, r = ms.linear_cross_entropy(h, w, t), ms.linear_cross_entropy_grad(h, w, t, grad_weight=False)
    assert torch.equal(s.lse, r.lse) and torch.equal(s.nll, r.nll)


def _inputs(n, v, d, dtype, seed, odd=False):
    """On the GPU; `odd`: rows at odd strides and addresses, so that they are packed."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    t16 = torch.bfloat16 if dtype == "bf16" else torch.float16
    w = (torch.randn(v, d, generator=g, device="cuda") * (2.5 / d ** 0.5)).to(t16)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    h = (torch.randn(n, d, generator=g, device="cuda") + 0.5 * w[t].float()).to(t16)
    t[torch.rand(n, generator=g, device="cuda") < 0.1] = -100
    h[t < 0] = float("nan")
    if odd:
        def lay(x):
            flat = torch.full((x.shape[0] * (d + 3) + 1,), float("nan"), dtype=t16, device="cuda")
            y = flat[1:].view(x.shape[0], d + 3)[:, :d]
            y.copy_(x)
            return y
        h, w = lay(h), lay(w)
    return h, w, t


def _check(r, h, w, t, *, dtype, cap=0.0, weights=None, step=None):
    """Every output of r that is not None against float64."""
    import torch
    n, d = h.shape
    v = w.shape[0]
    counted = t >= 0
    hf, wf = torch.where(counted[:, None], h, torch.zeros_like(h)).double(), w.double()
    at = t.clamp_min(0)
    g = counted.double() / counted.sum() if weights is None else weights.double() * counted
    wt, aw = wf.t().contiguous(), wf.abs()
    awt, sum_aw = aw.t().contiguous(), aw.sum(0)
    dw, adw = (torch.zeros(v, d, dtype=torch.float64, device="cuda") if r.grad_weight is not None else None for _ in "ab")
    loss = loss_tol = 0.0
    step = step or max(1, (1 << 27) // v)
    limit = 0.0
    for a in range(0, n, step):
        s = slice(a, min(n, a + step))
        z = torch.mm(hf[s], wt)
        lim = (d + 16) * 2.0 ** -24 * float(torch.mm(hf[s].abs(), awt).max())
        limit = max(limit, lim)
        y = torch.tanh(z / cap) * cap if cap else z
        k, rows = counted[s].double(), torch.arange(y.shape[0], device="cuda")
        lse = torch.logsumexp(y, 1)
        nll = (lse - y[rows, at[s]]) * k
        lse_tol = lim + 2.0 ** -20 * (1 + lse.abs())
        assert bool(((r.lse[s].double() - lse * k).abs() <= lse_tol).all()), f"lse at {a}"
        assert bool(((r.nll[s].double() - nll).abs() <= 2 * lse_tol).all()), f"nll at {a}"
        if r.loss is None:
            continue
        loss += float((g[s] * nll).sum())
        loss_tol += float((g[s].abs() * (2 * lse_tol + 2.0 ** -20 * nll.abs())).sum())
        y.sub_(lse[:, None]).exp_()
        y[rows, at[s]] -= 1.0
        y *= g[s][:, None]
        if cap:
            y *= 1.0 - torch.tanh(z / cap) ** 2
        del z
        share = 1.1 * U[dtype] + 2.0 ** -11 + (4 + (2 / cap if cap else 0)) * lim + (2.0 ** -18 if cap else 0)
        if r.grad_hidden is not None:
            dh = torch.mm(y, wf)
            tol = share * torch.mm(y.abs(), aw) + 1.01 * U[dtype] * dh.abs() + TINY[dtype]
            tol += 2.0 ** -37 * g[s].abs()[:, None] * sum_aw
            off = (r.grad_hidden[s].double() - dh).abs() / tol
            assert float(off.max()) <= 1.0, f"grad_hidden at {a}: {float(off.max()):.3g} of the tolerance"
        if dw is not None:
            yt = y.t().contiguous()
            dw += torch.mm(yt, hf[s])
            adw += torch.mm(yt.abs_(), hf[s].abs())
    if r.loss is not None:
        assert abs(float(r.loss) - loss) <= loss_tol + 1e-30, (float(r.loss), loss, loss_tol)
    if dw is not None:
        share = 1.1 * U[dtype] + 2.0 ** -11 + (4 + (2 / cap if cap else 0)) * limit + (2.0 ** -18 if cap else 0)
        tol = share * adw + 1.01 * U[dtype] * dw.abs() + TINY[dtype] + 2.0 ** -37 * (g.abs()[:, None] * hf.abs()).sum(0)
        off = (r.grad_weight.double() - dw).abs() / tol
        assert float(off.max()) <= 1.0, f"grad_weight: {float(off.max()):.3g} of the tolerance"


@pytest.mark.parametrize("dtype,cap,weighted,d,odd,only", [
    ("fp16", 0.0, False, 16, False, None), ("bf16", 6.0, True, 16, False, None), ("fp16", 6.0, True, 15, False, None),
    ("bf16", 0.0, True, 24, True, None), ("bf16", 0.0, False, 16, False, "grad_hidden"),
    ("bf16", 6.0, False, 9, True, "grad_weight"),
])
def test_pieces_in_every_form(dtype, cap, weighted, d, odd, only):
    """Three pieces of the tokens: weights, packed rows, a cap and one gradient alone count on from piece to piece."""
    import torch
    import muon_optimizer_step_amd as ms
    v = 1 << 20
    n = 2 * ms._lib.MUON_HEAD_PIECE_BYTES // (2 * v) + 188
    h, w, t = _inputs(n, v, d, dtype, seed=30 + d, odd=odd)
    weights = None
    if weighted:
        g = torch.Generator(device="cuda").manual_seed(31)
        weights = torch.randn(n, generator=g, device="cuda") * torch.exp(2 * torch.randn(n, generator=g, device="cuda")) / n
        weights[::17] = 0.0
    gu.say(f"[head large] pieces {n} x {v} x {d} {dtype} cap {cap} odd {odd} only {only}")
    kw = {k: False for k in ("grad_hidden", "grad_weight") if only and k != only}
    # tokens whose weight is zero but that count: their hidden states are finite
    r = ms.linear_cross_entropy_grad(h, w, t, softcap=cap, token_weights=weights, **kw)
    _check(r, h, w, t, dtype=dtype, cap=cap, weights=weights)


# (tokens, vocab, dim): exponentials beyond 192 MB, from each kernel of the logits that can have them, and beyond 1 GiB
PAST = [(20, 4000000, 8), (50, 2000003, 16), (100, 1200000, 16), (1100, 131072, 64), (8192, 80000, 32)]


@pytest.mark.parametrize("n,v,d", PAST)
@pytest.mark.parametrize("dtype,cap", [("bf16", 0.0), ("bf16", 6.0), ("fp16", 0.0), ("fp16", 6.0)])
def test_exponentials_past_the_caches(n, v, d, dtype, cap):
    import muon_optimizer_step_amd as ms
    h, w, t = _inputs(n, v, d, dtype, seed=40 + n)
    gu.say(f"[head large] past {n} x {v} x {d} {dtype} cap {cap}")
    _check(ms.linear_cross_entropy_grad(h, w, t, softcap=cap), h, w, t, dtype=dtype, cap=cap)


@pytest.mark.parametrize("cap,odd", [(0.0, False), (6.0, True)])
def test_scoring_in_pieces(cap, odd):
    """More than 2^32 logits."""
    import muon_optimizer_step_amd as ms
    n, v, d = 70000, 65537, 8
    h, w, t = _inputs(n, v, d, "bf16", seed=50, odd=odd)
    gu.say(f"[head large] scores {n} x {v} x {d} cap {cap} odd {odd}")
    _check(ms.linear_cross_entropy(h, w, t, softcap=cap), h, w, t, dtype="bf16", cap=cap)
