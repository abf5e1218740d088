"""GPU: the head's loss where a problem takes several pieces."""

import pytest

from tests import gpu_util as gu

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
