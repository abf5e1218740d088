"""Plain float64 oracle of the language-model head's loss and its gradients.

TEST INFRASTRUCTURE ONLY (imported by tests/).  Every step is one NumPy
expression in float64; nothing is shared with the HIP library.

    z = H W^T;  l = cap tanh(z / cap) (cap 0: l = z)
    lse_i = log sum_j exp l_ij;  nll_i = lse_i - l_i,t(i);  ignored tokens: 0
    g_i = weights_i, or 1 / (counted tokens);  loss = sum g_i nll_i
    P_ij = g_i (exp(l_ij - lse_i) - [j = t(i)]) (1 - (l_ij / cap)^2)
    dH = P W;  dW = P^T H
"""

from __future__ import annotations

import numpy as np


def head_loss(hidden, weight, targets, *, weights=None, ignore_index: int = -100, softcap: float = 0.0):
    """dict of nll, lse, loss, grad_hidden, grad_weight, and |P| |W|, |P|^T |H| (what rounding P is bounded by)."""
    h = np.asarray(hidden, dtype=np.float64).copy()
    w = np.asarray(weight, dtype=np.float64)
    t = np.asarray(targets)
    counted = t != ignore_index
    h[~counted] = 0.0                        # whatever an ignored token holds reaches nothing
    g = np.asarray(weights, dtype=np.float64) * counted if weights is not None else counted / max(1, counted.sum())
    z = h @ w.T
    lo = softcap * np.tanh(z / softcap) if softcap > 0 else z
    top = lo.max(axis=1)
    lse = top + np.log(np.exp(lo - top[:, None]).sum(axis=1))
    rows = np.arange(len(t))
    at = np.where(counted, t, 0)
    nll = np.where(counted, lse - lo[rows, at], 0.0)
    p = np.exp(lo - lse[:, None])
    p[rows, at] -= 1.0
    p *= g[:, None]
    if softcap > 0:
        p *= 1.0 - (lo / softcap) ** 2
    return {"nll": nll, "lse": np.where(counted, lse, 0.0), "loss": float((g * nll).sum()),
            "grad_hidden": p @ w, "grad_weight": p.T @ h, "abs_hidden": np.abs(p) @ np.abs(w),
            "abs_weight": np.abs(p).T @ np.abs(h), "abs_logit": float((np.abs(h) @ np.abs(w).T).max())}
