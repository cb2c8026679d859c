"""The 8-bit integer calls refuse bad arguments before touching the device
(include/wq.h, "8-bit integer linears"); the binding refuses bad tensors before
any pointer reaches the C ABI."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def wq():
    import quantized_gemm_wq_b200 as wq
    return wq


P = 1 << 20          # a non-null, 16-byte aligned fake address: never dereferenced
BIG = 1 << 31


def test_quantize_refusals(wq):
    q = wq.lib.wq_quantize_i8
    ok = dict(x=P, t=0, R=4, K=64, ldx=64, c=P, ldc=64, s=P)

    def call(**kw):
        a = {**ok, **kw}
        return q(a["x"], a["t"], a["R"], a["K"], a["ldx"], a["c"], a["ldc"], a["s"], None)

    for k in ("x", "c", "s"):
        assert call(**{k: None}) == wq.WQ_ERR_NULL
    for t in (-1, 3):
        assert call(t=t) == wq.WQ_ERR_TYPE
    for kw in (dict(R=0), dict(K=0), dict(R=-1), dict(R=BIG, ldx=64), dict(K=131072, ldx=131072, ldc=131072)):
        assert call(**kw) == wq.WQ_ERR_SHAPE, kw
    for kw in (dict(ldx=63), dict(ldc=48), dict(ldc=72), dict(ldx=BIG), dict(ldc=BIG), dict(ldx=0), dict(ldx=-64)):
        assert call(**kw) == wq.WQ_ERR_STRIDE, kw
    for kw in (dict(x=P + 1), dict(t=2, x=P + 2), dict(c=P + 8), dict(s=P + 2)):
        assert call(**kw) == wq.WQ_ERR_ALIGN, kw
    # what the rules allow is refused for the missing device alone
    for kw in (dict(), dict(x=P + 2), dict(t=2, x=P + 4, s=P + 4), dict(ldx=65), dict(K=131071, ldx=131071, ldc=131072)):
        if not torch.cuda.is_available():
            assert call(**kw) in (wq.WQ_ERR_CUDA, wq.WQ_ERR_UNSUPPORTED_DEVICE), kw


@pytest.mark.parametrize("gated", [False, True])
def test_product_refusals(wq, gated):
    ok = dict(x=P, ldx=64, xs=P, M=4, N=8, K=64, w=P, ws=P, u=P, us=P, ldw=64, act=0, y=P, t=0, ldy=8)

    def call(**kw):
        a = {**ok, **kw}
        if gated:
            return wq.lib.wq_gated_i8(a["x"], a["ldx"], a["xs"], a["M"], a["N"], a["K"], a["w"], a["ws"], a["u"],
                                      a["us"], a["ldw"], a["act"], a["y"], a["t"], a["ldy"], None)
        return wq.lib.wq_gemm_i8(a["x"], a["ldx"], a["xs"], a["M"], a["N"], a["K"], a["w"], a["ldw"], a["ws"],
                                 a["y"], a["t"], a["ldy"], None)

    for k in ("x", "xs", "w", "ws", "y") + (("u", "us") if gated else ()):
        assert call(**{k: None}) == wq.WQ_ERR_NULL, k
    for kw in (dict(t=3), dict(t=-1)) + ((dict(act=3), dict(act=-1)) if gated else ()):
        assert call(**kw) == wq.WQ_ERR_TYPE, kw
    for kw in (dict(M=0), dict(N=0), dict(K=0), dict(M=BIG), dict(N=BIG, ldy=BIG - 1), dict(M=-3),
               dict(K=131072, ldx=131072, ldw=131072)):
        assert call(**kw) == wq.WQ_ERR_SHAPE, kw
    for kw in (dict(ldx=48), dict(ldw=48), dict(ldy=7), dict(ldx=72), dict(ldw=65), dict(ldx=BIG), dict(ldw=BIG),
               dict(ldy=BIG)):
        assert call(**kw) == wq.WQ_ERR_STRIDE, kw
    for kw in (dict(x=P + 8), dict(w=P + 4), dict(xs=P + 1), dict(ws=P + 2), dict(y=P + 1), dict(t=2, y=P + 2)) + (
            (dict(u=P + 8), dict(us=P + 2)) if gated else ()):
        assert call(**kw) == wq.WQ_ERR_ALIGN, kw
    for kw in (dict(), dict(y=P + 2), dict(K=63), dict(K=1, N=1, ldy=1), dict(K=131071, ldx=131072, ldw=131072)):
        if not torch.cuda.is_available():
            assert call(**kw) in (wq.WQ_ERR_CUDA, wq.WQ_ERR_UNSUPPORTED_DEVICE), kw


def test_status_strings(wq):
    assert "type" in wq.wq_status_string(wq.WQ_ERR_TYPE)
    assert "stride" in wq.wq_status_string(wq.WQ_ERR_STRIDE)


def test_binding_checks_tensors(wq):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    c = torch.zeros(2, 64, dtype=torch.int8)
    s = torch.zeros(2)
    with pytest.raises(ValueError):
        wq.wq_quantize_i8(x)                                 # host tensor
    with pytest.raises(ValueError):
        wq.wq_quantize_i8(x.double())                        # type
    with pytest.raises(ValueError):
        wq.wq_gemm_i8(c, s, c, s)                            # host tensors
    with pytest.raises(ValueError):
        wq.wq_gemm_i8(c.float(), s, c, s)                    # not codes
    with pytest.raises(ValueError):
        wq.wq_gated_i8(c, s, c, s, c, s, act="tanh")         # unknown activation
    with pytest.raises(ValueError):
        wq.wq_gated_i8(c, s, c, s, c, s)                     # host tensors


def test_enums_match_the_header(wq):
    """wq_type and wq_act values of the header against the binding's tables."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "wq.h")).read()
    enum = {k: int(v) for k, v in re.findall(r"(WQ_(?:TYPE|ACT|ERR)_[A-Z0-9_]+)\s*=\s*(\d+)", src)}
    assert {torch.bfloat16: enum["WQ_TYPE_BF16"], torch.float16: enum["WQ_TYPE_F16"],
            torch.float32: enum["WQ_TYPE_F32"]} == wq._TYPES
    assert {"silu": enum["WQ_ACT_SILU"], "gelu": enum["WQ_ACT_GELU"],
            "gelu_tanh": enum["WQ_ACT_GELU_TANH"]} == wq._ACTS
    assert wq.WQ_ERR_TYPE == enum["WQ_ERR_TYPE"] and wq.WQ_ERR_STRIDE == enum["WQ_ERR_STRIDE"]
    assert ctypes.sizeof(ctypes.c_int) == 4      # how the binding passes both
