"""The weight-only tensor-core kernels where bounded waits run out: the test build,
whose pipeline waits have no time, on batches that the TMEM GEMV, the swap-AB GEMM and
the prefill GEMM (one and two launches) take.  Each wait finds its stage landed or gives up, the
copies and MMAs in flight are seen out, and right after, in the same process and
context, the library proper computes what it did before."""
from __future__ import annotations

import ctypes
import multiprocessing as mp
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _child(q, M, N, K, bits, group):
    import sys
    sys.path.insert(0, ROOT)
    try:
        import torch

        import quantized_gemm_wq_b200 as wq
        import wq_inputs
        short = ctypes.CDLL(os.path.join(ROOT, "quantized_gemm_wq_b200", "libwq_shortwait.so"))
        for name in ("wq_gemm", "wq_last_device_error"):
            getattr(short, name).argtypes = getattr(wq.lib, name).argtypes
            getattr(short, name).restype = getattr(wq.lib, name).restype
        W = torch.from_numpy(wq_inputs.weight_f16(62, 0, N, K)).cuda()
        c, s, z = wq.wq_quantize_rtn(W, bits, group)
        x = wq_inputs.activations_bf16(62, M, M, K).cuda()
        want = wq.wq_gemm(x, c, s, z, bits, group, N, K)
        assert wq.wq_last_device_error() == 0
        res = []
        for _ in range(5):
            y = torch.empty_like(want)
            st = short.wq_gemm(x.data_ptr(), M, N, K, c.data_ptr(), s.data_ptr(), z.data_ptr(), bits, group,
                               y.data_ptr(), None)
            err, then = short.wq_last_device_error(), short.wq_last_device_error()
            after = bool(torch.equal(wq.wq_gemm(x, c, s, z, bits, group, N, K), want)) and wq.wq_last_device_error() == 0
            res.append((st, err, then, after, err == 8 or bool(torch.equal(y, want))))
        q.put(res)
    except Exception as e:  # noqa: BLE001
        q.put(repr(e))


@pytest.mark.parametrize("M,N,K,bits,group", [(16, 4096, 4096, 4, 128), (12, 1024, 2048, 3, 0), (64, 1024, 4096, 4, 128),
                                              (130, 600, 2048, 8, 128), (256, 512, 2048, 4, 128),
                                              (300, 777, 1024, 2, 0), (2048, 5120, 1024, 4, 128)])
def test_waits_that_run_out(M, N, K, bits, group):
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    pr = ctx.Process(target=_child, args=(q, M, N, K, bits, group))
    pr.start()
    res = q.get(timeout=300)
    pr.join(60)
    assert isinstance(res, list), res
    for st, err, then, after, right in res:
        assert st == 0 and err in (0, 8) and then == 0 and after and right, res
