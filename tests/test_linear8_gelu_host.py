"""The constants of gelu's tail in csrc/blocks8.hip on the host: the fit that they come from, repeated, and what they reach.

erfc(z) = exp(-z^2) t P(t) with t = 1 / (1 + p z): P has nine coefficients, fitted for the least largest relative error of t P(t) against
exp(z^2) erfc(z) over 0 <= z <= 13.5, by least squares whose weights grow where the error is large.
"""

import os
import re

import numpy as np
import pytest

scipy_special = pytest.importorskip("scipy.special")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAR = 13.5


def _constants():
    text = open(os.path.join(ROOT, "muon_optimizer_step_amd", "csrc", "blocks8.hip")).read()
    body = text[text.index("inline Gelu gelu_parts"):]
    body = body[:body.index("return {")]
    p = float(re.search(r"\* (0\.\d+)f, a, 1\.f", body).group(1))
    return p, [float(x) for x in re.findall(r"float q = (-?[\d.]+)f", body) + re.findall(r"fmaf\(q, t, (-?[\d.]+)f\)", body)]


def _fit(p, degree):
    """(coefficients from the constant on, largest relative error) of the best P for this p."""
    low = 1 / (1 + p * FAR)
    t = (np.cos(np.pi * (np.arange(4000) + 0.5) / 4000) + 1) / 2 * (1 - low) + low
    want = scipy_special.erfcx((1 / t - 1) / p) / t
    powers, weight = np.vander(t, degree + 1, increasing=True) / want[:, None], np.ones(len(t))
    for _ in range(300):
        c = np.linalg.lstsq(powers * np.sqrt(weight)[:, None], np.sqrt(weight), rcond=None)[0]
        error = np.abs(powers @ c - 1)
        weight *= error / error.max() + 1e-3
        weight /= weight.mean()
    return c, error.max()


def _errors(p, coefficients, number):
    """Relative errors over z, every operation rounded to `number`."""
    z = np.concatenate([np.linspace(0, 1, 100001), np.linspace(1, FAR, 200001)]).astype(number)
    t = (1 / (z.astype(np.float64) * number(p) + 1).astype(number).astype(np.float64)).astype(number)
    q = np.full_like(t, number(coefficients[0]))
    for c in coefficients[1:]:
        q = (q.astype(np.float64) * t + np.float64(number(c))).astype(number)      # fused: exact in 64 bits but for their last digits
    return (q * t).astype(number).astype(np.float64) / scipy_special.erfcx(z.astype(np.float64)) - 1


def test_the_fit():
    p, coefficients = _constants()
    assert len(coefficients) == 9
    fitted, error = _fit(p, 8)
    assert error < 3.9e-8
    # p is the best to its digits: 2 % to either side is worse
    assert _fit(p * 1.02, 8)[1] > error and _fit(p * 0.98, 8)[1] > error
    # the constants are the fitted ones to float32's digits: as polynomials the two differ by half a step of each
    t = np.linspace(1 / (1 + p * FAR), 1, 2001)
    two = [sum(c * t ** k for k, c in enumerate(x)) for x in (fitted, coefficients[::-1])]
    assert np.abs(two[0] / two[1] - 1).max() < 1.2e-7


def test_what_they_reach():
    p, coefficients = _constants()
    assert np.abs(_errors(p, coefficients, np.float64)).max() < 1.0e-7
    assert np.abs(_errors(p, coefficients, np.float32)).max() < 3.5e-7
