"""The polynomial that stands for erfc in the gelu of wq_gated_i8: its coefficients as
csrc/i8.cuh holds them, against math.erfc over the range where exp(-z^2) is not 0 in fp32."""
import math
import os
import re
from fractions import Fraction

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_gemm_wq_b200", "csrc",
                   "i8.cuh")
U = 2.0 ** -24


def _fit():
    """(p, coefficients, highest power first) with the values that fp32 holds."""
    src = open(SRC).read()
    body = src[src.index("float erfc_tail(float t)"):]
    body = body[:body.index("}")]
    coeffs = [float(c) for c in re.findall(r"(-?\d\.\d+)f", body)]
    p = float(re.search(r"t = 1 / \(1 \+ ([\d.]+) z\)", src).group(1))
    scale = float(re.search(r"fmaf_rn\(fabsf\(g\), ([\d.]+)f, 1\.0f\)", src).group(1))
    assert abs(scale - p * math.sqrt(0.5)) < 1e-15
    assert len(coeffs) == 9
    for c in coeffs:
        assert float(np.float32(c)) == c        # written as fp32 holds them
    return p, coeffs


def test_fit_error():
    """erfc(z) = exp(-z^2) t P(t), t = 1 / (1 + p z), to under one unit of 2^-24 of its value: the fit by
    itself, in 64 bits."""
    p, coeffs = _fit()
    z = np.linspace(0.0, 10.2, 20401)           # exp(-10.2^2) is below half of fp32's smallest number
    assert math.exp(-10.2 ** 2) < 2.0 ** -150
    t = 1.0 / (1.0 + p * z)
    v = np.zeros_like(t)
    for c in coeffs:
        v = v * t + c
    ref = np.array([math.erfc(x) for x in z])
    # exp(-z^2) in exact exponents: z^2 is rounded by 2^-53 of up to 104, 1.2e-14 of the value
    err = np.abs(t * v * np.exp(-z * z) / ref - 1.0)
    assert err.max() < U, err.max()


def test_fit_steps_in_fp32():
    """The polynomial's nine fp32 steps (one rounding each) stay within 2 units of 2^-24 of its value."""
    p, coeffs = _fit()
    t = (1.0 / (1.0 + p * np.linspace(0.0, 10.2, 2001))).astype(np.float32)
    v = np.full(t.shape, np.float32(coeffs[0]))
    for c in coeffs[1:]:
        v = np.array([np.float32(float(Fraction(float(a)) * Fraction(float(b)) + Fraction(c))) for a, b in zip(v, t)])
    w = np.zeros(t.shape)
    for c in coeffs:
        w = w * t.astype(np.float64) + c
    assert np.abs(v / w - 1.0).max() < 2 * U
