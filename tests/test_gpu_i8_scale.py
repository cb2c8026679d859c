"""The scale of wq_quantize_i8 is max|x| times fp32(1/127), one rounding: rows whose
rounded quotient max|x| / 127 is another number, and rows whose scale is rounded to 0."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from i8_util import quantize_ref, wq

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _maxima(dtype):
    """Maxima of the type for which the two scales differ."""
    rng = np.random.default_rng(21)
    a = torch.from_numpy(np.exp(rng.normal(0, 1, 20000))).to(dtype).float().numpy()
    prod = a * np.float32(1.0 / 127.0)
    quot = (a.astype(np.float64) / 127.0).astype(np.float32)
    return a, prod, quot


@pytest.mark.parametrize("dtype", TYPES)
def test_the_two_scales_differ_as_stated(dtype):
    a, prod, quot = _maxima(dtype)
    step = np.abs(prod.view(np.int32) - quot.view(np.int32))
    assert step.max() == 1 and 0.02 < (step > 0).mean() < 0.1
    off = np.abs(prod.astype(np.float64) * 127.0 / a - 1.0).max()
    # fp32(1/127) is 3.8e-9 of its value away from 1/127, and the product rounds by up to 2^-24 of it
    assert off < 6.4e-8


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_scale_is_the_product(dtype):
    a, prod, quot = _maxima(dtype)
    a = a[prod != quot][:300]
    rng = np.random.default_rng(22)
    x = torch.from_numpy(rng.uniform(-1, 1, (len(a), 96)) * a[:, None]).to(dtype)
    x[:, 17] = torch.from_numpy(-a).to(dtype)
    q, s = wq().wq_quantize_i8(x.cuda())
    rq, rs = quantize_ref(x.double().numpy())
    assert (rs == a * np.float32(1.0 / 127.0)).all() and (rs != (a.astype(np.float64) / 127.0).astype(np.float32)).all()
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


@pytest.mark.gpu
def test_scale_that_rounds_to_zero():
    step = 2.0 ** -149
    x = torch.tensor([[63.0, -5.0], [64.0, -5.0], [190.0, 1.0], [0.0, 0.0]]).double() * step
    q, s = wq().wq_quantize_i8(x.float().cuda())
    assert (s.double() / step).tolist() == [0.0, 1.0, 1.0, 0.0]
    assert q.tolist() == [[0, 0], [64, -5], [127, 1], [0, 0]]
