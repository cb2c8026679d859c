"""The activations of wq_gated_i8 by themselves: the gate's scales carry g exactly
(one product of 1 and 1), u = 1, so h is act(g) and nothing else is rounded."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from i8_util import U, assert_rounds_to, codes, scales, wq

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh"]
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _act(g, act, M, dtype):
    """h of M equal tokens for the gate values g."""
    N = len(g)
    x = torch.zeros(M, 16, dtype=torch.int8, device="cuda")
    x[:, 0] = 1
    w = torch.zeros(N, 16, dtype=torch.int8, device="cuda")
    w[:, 0] = 1
    return wq().wq_gated_i8(x, torch.ones(M, device="cuda"), w, torch.from_numpy(g).cuda(), w,
                            torch.ones(N, device="cuda"), act=act, dtype=dtype)


def _grid():
    return np.concatenate([np.linspace(-16, 16, 30011), np.linspace(-1, 1, 4001), np.linspace(-130, -60, 9001),
                           np.linspace(-120, 120, 4001), np.geomspace(1e-38, 1e38, 2001), -np.geomspace(1e-38, 1e38, 2001),
                           [0.0, -0.0, 1e-42, -1e-42]]).astype(np.float32)


# tokens for each kernel: warp MMAs, split (one and three token tiles of 32), pair
KERNELS = [1, 8, 9, 40, 96, 128, 300]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
def test_activation_is_one_function_in_every_kernel(act, dtype):
    """The same gate values through every kernel: the same bits, one token or 300."""
    g = _grid()
    want = _act(g, act, 1, dtype)
    for M in KERNELS[1:]:
        h = _act(g, act, M, dtype)
        assert torch.equal(h.view(torch.int16 if dtype != torch.float32 else torch.int32),
                           want.expand(M, -1).contiguous().view(torch.int16 if dtype != torch.float32 else torch.int32)), M


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
def test_gated_rows_do_not_depend_on_the_batch(act, dtype):
    """The same tokens, alone and in batches that other kernels take: the same bits."""
    rng = np.random.default_rng(12)
    N, K = 1300, 333
    x, _ = codes(rng, 600, K)
    xs, _ = scales(rng, 600)
    w, _ = codes(rng, N, K)
    ws, _ = scales(rng, N)
    u, _ = codes(rng, N, K)
    us, _ = scales(rng, N)
    ws *= 1.0 / (74.0 ** 2 * K ** 0.5 * 1e-3)           # gate values of unit size, and their spread
    us *= 1e-3
    full = wq().wq_gated_i8(x, xs, w, ws, u, us, act=act, dtype=dtype)
    assert torch.isfinite(full).all() and (full != 0).float().mean() > 0.5
    for m in (1, 2, 8, 9, 16, 33, 64, 128, 129, 257):
        h = wq().wq_gated_i8(x[5:5 + m], xs[5:5 + m], w, ws, u, us, act=act, dtype=dtype)
        assert torch.equal(h, full[5:5 + m]), m


def _reference(g, act):
    """act(g) and |t|, the size of the exponential's argument, in 64 bits."""
    gt = torch.from_numpy(g.astype(np.float64))
    if act == "silu":
        return (gt * torch.special.expit(gt)).numpy(), gt.abs().numpy()
    if act == "gelu":
        return (0.5 * gt * torch.special.erfc(-gt / math.sqrt(2.0))).numpy(), (gt * gt / 2).numpy()
    t = 2.0 * math.sqrt(2.0 / math.pi) * (gt + 0.044715 * gt ** 3)
    return (gt * torch.special.expit(t)).numpy(), t.abs().numpy()


def _units(g, v, act, dtype):
    """The error of act(g) before the rounding to the result's type, in units of U = 2^-24 of its value.

    silu, gelu_tanh = g e / (1 + e): the exponential, 2 steps = 4 (expf for fp32 results; the hardware's 2^x,
    with 2.4 v from its argument, for 16-bit ones), g e 1, 1 + e 1, its reciprocal 1 step = 2, the product 1
    (far below zero fewer: a constant factor in the reciprocal's place); t of gelu_tanh 4 |t|: two constants,
    g^2, an fma, a product.  gelu: the fit 1 and its steps 2, e t, the fit's factor and g 3, t = 1 / (1 + p z)
    with its constant, fma and reciprocal at most 3.4, of which erfc feels up to 2.35 times as much: 8;
    exp(-g^2 / 2) 4, and v from its argument (2.4 v more with the hardware's).
    Above zero an error of the exponential's counts with e / (1 + e), and v e^-v < 1."""
    v = np.where(g < 0, v, 1.0)
    if dtype == torch.float32:
        return {"silu": 9 + 0 * v, "gelu": 18 + v, "gelu_tanh": 9 + 4 * v}[act]
    return {"silu": 9 + 2.4 * v, "gelu": 18 + 3.4 * v, "gelu_tanh": 9 + 6.4 * v}[act]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_activation_error(act, dtype, M):
    """The activation within the error that the header states, down to where its value leaves fp32's
    normal range; under it within 2^-140."""
    g = _grid()
    g = g[np.abs(g) <= 1e4]
    ref, v = _reference(g, act)
    err = np.abs(ref) * _units(g, v, act, dtype) * U * 1.01 + 2.0 ** -140
    assert_rounds_to(_act(g, act, M, dtype)[M - 1:], ref[None], err[None], f"{act} {dtype}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_gates_at_the_ends(act, dtype, M):
    """Gates whose square or cube leaves fp32, infinite ones and NaN: the limit above zero and below,
    NaN for minus infinity (a product of it and 0) and for NaN."""
    inf = float("inf")
    g = np.array([3e19, 3e38, inf, -3e19, -3e38, -200.0, -inf, np.nan, 0.0, -0.0], np.float32)
    h = _act(g, act, M, dtype)[M - 1]
    top = torch.from_numpy(g[:3]).to(dtype).cuda()
    assert torch.equal(h[:3], top)
    assert (h[3:6] == 0).all() and torch.isnan(h[6:8]).all()
    assert (h[8:] == 0).all() and torch.signbit(h[8:]).tolist() == [False, True]
