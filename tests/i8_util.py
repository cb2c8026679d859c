"""A plain 64-bit statement of the 8-bit integer linears for the tests, the
inputs they share, and the bounds their results are held to."""
from __future__ import annotations

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SMALLEST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}   # subnormal step
U = 2.0 ** -24       # half a step of fp32


def wq():
    import quantized_gemm_wq_b200 as m
    return m


def quantize_ref(x: np.ndarray):
    """codes, scales of float64 rows that hold values of a narrower type."""
    with np.errstate(all="ignore"):
        a = np.abs(x).max(axis=1)
        s = a.astype(np.float32) * np.float32(1.0 / 127.0)
        bad = ~np.isfinite(x).all(axis=1)
        s[bad] = np.nan
        s64 = s.astype(np.float64)[:, None]
        q = np.rint(np.divide(x, s64, out=np.zeros_like(x), where=s64 > 0))
    q = np.where(bad[:, None], 0.0, np.clip(q, -127, 127))
    return q.astype(np.int8), s


def product(x, w):
    """The exact sums (float64 holds every one: below 2^31)."""
    return x.astype(np.float64) @ w.astype(np.float64).T


def scaled_f32(acc, xs, ws):
    """The three fp32 roundings that wq.h defines, in numpy."""
    with np.errstate(all="ignore"):
        return (acc.astype(np.float32) * xs[:, None].astype(np.float32)) * ws[None, :].astype(np.float32)


def gated_ref(accg, accu, xs, gs, us, act):
    """h in 64 bits, and the bound on |h_fp32 - h| before the last rounding.

    g and u carry three roundings each (3 U relative).  d(act)/act <= c |dg/g|
    with c = 1 + |g| (silu), 2 + g^2 (gelu: |z erfc'(z) / erfc(z)| <= 1 + 2 z^2
    at z = |g| / sqrt 2, one more for the factor g) and 1 + 3 |t| (gelu_tanh:
    |dt/t| <= 3 |dg/g|).  The activation itself, in units of U: the hardware's
    exponential of v, 2 + 1.173 |v| steps (the CUDA guide's bound) = 4 + 2.4 |v|,
    the sum 1, its division 2 steps = 4, t's own evaluation 8 |t|; gelu's
    erfc: the fit 1 (6e-8), its nine steps and three products 9 as simulated, t's
    division 4, and exp(-g^2 / 2) 4 + 1.2 g^2, its argument's rounding g^2 / 2:
    at most 18 + 2 g^2.  The product with u: 3 + 1.
    Far below zero the activation leaves fp32's normal range: where 1 + exp(-g)
    (or exp(-t)) passes 2^126 the hardware's quotient is 0, for a true |act| <
    |g| 2^-126, and one under 2^-126 may be flushed: together at most
    (|g| + 1) 2^-126 |u|, and 2^-126 for the product's own underflow."""
    import math
    import torch as t
    g = accg * xs[:, None].astype(np.float64) * gs[None, :].astype(np.float64)
    u = accu * xs[:, None].astype(np.float64) * us[None, :].astype(np.float64)
    gt = t.from_numpy(g)
    if act == "silu":
        a = (gt * t.sigmoid(gt)).numpy()
        units = 3 * (1 + np.abs(g)) + 4 + 2.4 * np.abs(g) + 1 + 4
    elif act == "gelu":
        a = (0.5 * gt * t.special.erfc(-gt / math.sqrt(2.0))).numpy()
        units = 3 * (2 + g * g) + 18 + 2 * g * g
    else:
        tt = 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
        a = g / (1.0 + np.exp(-np.clip(tt, -700, 700)))
        units = 3 * (1 + 3 * np.abs(tt)) + 4 + 2.4 * np.abs(tt) + 1 + 4 + 8 * np.abs(tt)
    h = a * u
    return h, np.abs(h) * (units + 4) * U * 1.01 + 2.0 ** -126 + (np.abs(g) + 1) * 2.0 ** -126 * np.abs(u)


def assert_rounds_to(y: torch.Tensor, ref: np.ndarray, err: np.ndarray, what=""):
    """|y - ref| <= err + half a step of y's type (relative, or of its subnormals);
    infinite only where ref, err away at most, passes the half step above the largest value."""
    f = torch.finfo(y.dtype)
    y64 = y.double().cpu().numpy()
    top = f.max * (1 + HALF_STEP[y.dtype] / 2)      # max is (2 - eps) 2^e: half a step is a quarter eps of it
    over = np.isinf(y64) & (np.sign(y64) == np.sign(ref)) & (np.abs(ref) + err >= top * (1 - HALF_STEP[y.dtype]))
    with np.errstate(invalid="ignore"):
        d = np.where(over, 0.0, np.abs(y64 - ref))
    lim = err + HALF_STEP[y.dtype] * (np.abs(ref) + err) + 0.5 * SMALLEST[y.dtype]
    bad = ~(d <= lim)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; first {i}: {y[i].item()} for {ref[i]}, "
                             f"off by {d[i]}, allowed {lim[i]}")


def codes(rng, rows, K, pad=0, lo=-127):
    """int8 codes as the first columns of a wider buffer (16-byte rows), the rest garbage; and as numpy."""
    ld = (K + 15) // 16 * 16 + pad
    wide = rng.integers(-128, 128, (rows, ld), dtype=np.int8)
    c = rng.integers(lo, 128, (rows, K), dtype=np.int8)
    wide[:, :K] = c
    return torch.from_numpy(wide).cuda()[:, :K], c


def scales(rng, n):
    s = np.exp(rng.normal(-4.0, 1.0, n)).astype(np.float32)
    return torch.from_numpy(s).cuda(), s
