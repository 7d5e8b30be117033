"""CPU check of the Gaussian tail behind GELU in the 16-bit operators
(csrc/gemm16.cuh): erfc(z) / 2 as exp(-z^2) times a polynomial in
t = 1 / (1 + z / 2).  The fit is made again here by a linear program, and the
form is evaluated in fp32 over its whole range."""
import os
import re

import numpy as np
import pytest

import w4a4_quantized_gemm_smooth_b200 as S

special = pytest.importorskip("scipy.special")
Z_MAX = 9.4                          # exp(-z^2) leaves fp32 there


def coefficients():
    """Of t, t^2, ..., as the source holds them."""
    path = os.path.join(os.path.dirname(S.__file__), "csrc", "gemm16.cuh")
    text = open(path).read()
    body = text[text.index("GaussTail gauss_tail("):]
    body = body[:body.index("return g;")]
    c = [float(v) for v in re.findall(r"c\((-?[0-9.e-]+)f\)", body)]
    assert len(c) == 7
    return np.array(c[::-1])


def test_coefficients_are_the_minimax_fit():
    optimize = pytest.importorskip("scipy.optimize")
    z = np.linspace(0, Z_MAX, 4001)
    t, h = 1 / (1 + z / 2), special.erfc(z) / 2
    terms = np.exp(-z * z)[:, None] * t[:, None] ** np.arange(1, 8)
    weight = np.minimum(1e-7, 2e-5 * h)[:, None]        # absolute error over 1e-7, relative over 2e-5
    a, b = terms / weight, h / weight[:, 0]
    # least d with |a c - b| <= d
    d = -np.ones((len(z), 1))
    fit = optimize.linprog([0] * 7 + [1], A_ub=np.block([[a, d], [-a, d]]), b_ub=np.concatenate([b, -b]),
                           bounds=[(None, None)] * 7 + [(0, None)], method="highs")
    assert fit.status == 0
    c = coefficients()
    assert np.abs(a @ c - b).max() <= 1.03 * fit.x[7]
    assert np.abs(c - fit.x[:7]).max() <= 1e-5


def test_tail_in_fp32():
    """The stated bounds, with every step rounded to fp32 (the approximate
    reciprocal and exponential add a step or two of their own)."""
    f = np.float32
    x = np.concatenate([np.linspace(0, 13.2, 200001), np.geomspace(1e-8, 1, 2000)]).astype(f)
    z = x * f(0.70710678)
    t = f(1) / (z * f(0.5) + f(1))
    e = np.exp2(((x * f(-0.72134752)) * x).astype(np.float64)).astype(f)
    c = coefficients().astype(f)
    p = t * c[6] + c[5]
    for k in (4, 3, 2, 1, 0):
        p = (p * t + c[k]).astype(f)
    h = (p * t * e).astype(np.float64)
    want = special.erfc(x.astype(np.float64) * 0.5 ** 0.5) / 2
    live = want > 2.0 ** -126
    assert np.abs(h - want).max() <= 2e-7
    assert np.abs(h / want - 1)[live].max() <= 1.5e-5
