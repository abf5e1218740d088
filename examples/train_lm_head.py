"""A training step put together from the library's pieces, on a small next-token model.

    token -> embedding -> h + tanh(h W^T) -> scaled to unit root mean square, times a gain -> head

* the head's loss and its gradients: PreparedLinearCrossEntropy (the logits are never kept);
* the body's gradients: torch autograd, started from the loss's grad_hidden;
* W, a hidden matrix: PreparedMuonStep;
* the embedding, the head and the gain: one PreparedAdamW8 call, with 8-bit states for the two matrices and 32-bit
  ones for the gain; it also writes the bfloat16 copies that the next forward pass reads.

The data is a synthetic Markov chain in which each token has four successors, so the loss can fall to log 4 = 1.39.

    python examples/train_lm_head.py [--vocab 4096] [--dim 512] [--tokens 16384] [--steps 100]
"""

from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import muon_optimizer_step_amd as ms  # noqa: E402

COEFFS = [(3.4445, -4.7750, 2.0315)] * 5


def train(vocab=4096, dim=512, tokens=16384, steps=100, seed=0, masked=0.1, log=None):
    """Runs `steps` steps; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    successors = torch.randint(0, vocab, (vocab, 4), generator=g, device="cuda")

    emb, head = randn(vocab, dim), 0.02 * randn(vocab, dim)
    w, gain = randn(dim, dim) / dim ** 0.5, torch.ones(dim, device="cuda")
    emb16, head16 = emb.bfloat16().requires_grad_(), head.bfloat16()
    w.requires_grad_()
    gain.requires_grad_()

    # buffers that the prepared calls keep: hidden states, targets, gradients
    hidden = torch.empty(tokens, dim, dtype=torch.bfloat16, device="cuda")
    targets = torch.empty(tokens, dtype=torch.int64, device="cuda")
    loss = ms.PreparedLinearCrossEntropy(hidden, head16, targets, grads=True, ignore_index=-100)
    grads = [torch.empty_like(emb16), loss.result.grad_weight, torch.empty_like(gain)]
    states = [ms.AdamW8State.zeros_like(emb), ms.AdamW8State.zeros_like(head),
              (torch.zeros_like(gain), torch.zeros_like(gain))]
    adamw = ms.PreparedAdamW8([emb, head, gain.detach()], grads, states, copies=[emb16.detach(), head16, None])
    w_grad, momentum = torch.empty_like(w), torch.zeros(dim, dim, device="cuda")
    muon = ms.PreparedMuonStep([w.detach()], [w_grad], [momentum])

    losses = []
    for step in range(1, steps + 1):
        x = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        pick = torch.randint(0, 4, (tokens, 1), generator=g, device="cuda")
        targets.copy_(successors[x].gather(1, pick)[:, 0])
        targets[torch.rand(tokens, generator=g, device="cuda") < masked] = -100     # tokens that are not learned from

        h = torch.nn.functional.embedding(x, emb16).float()
        h = h + torch.tanh(h @ w.T)
        out = (h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * gain).bfloat16()
        hidden.copy_(out.detach())
        r = loss()                                          # loss, grad_hidden, grad_weight of the head
        d_emb, d_w, d_gain = torch.autograd.grad(out, (emb16, w, gain), r.grad_hidden)
        for dst, src in ((grads[0], d_emb), (grads[2], d_gain), (w_grad, d_w)):
            dst.copy_(src)
        muon(lr=0.02, momentum=min(0.95, 0.85 + 0.002 * step), weight_decay=0.0, coeffs=COEFFS)
        adamw(lr=0.01, betas=(0.9, 0.99), weight_decay=0.0, step=step, seed=seed)
        losses.append(r.loss.clone())
        if log and (step % 10 == 0 or step == 1):
            log(f"step {step:4d}  loss {float(r.loss):.4f}")
    return [float(x) for x in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("vocab", 4096), ("dim", 512), ("tokens", 16384), ("steps", 100)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    t = time.perf_counter()
    losses = train(a.vocab, a.dim, a.tokens, a.steps, log=lambda s: print(s, flush=True))
    print(f"{a.steps} steps in {time.perf_counter() - t:.2f} s: loss {losses[0]:.3f} -> {losses[-1]:.3f}")


if __name__ == "__main__":
    main()
