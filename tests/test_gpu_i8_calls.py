"""The 8-bit integer calls as programs make them: one behind another on a
stream without waiting, beside the library's other calls, from two threads, on
matrices past 2^32 bytes and elements, and where a bounded wait runs out."""
from __future__ import annotations

import ctypes
import multiprocessing as mp
import os
import threading

import numpy as np
import pytest
import torch

import wq_inputs
from i8_util import codes, product, quantize_ref, scaled_f32, scales, wq

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("M", [1, 16, 100, 300])
def test_weights_rewritten_just_before_the_product(M):
    """Each product reads the codes that the call right before it wrote into the same
    buffer (the product's kernel starts, and touches the weights' lines, before that call ends)."""
    m = wq()
    rng = np.random.default_rng([1, M])
    N, K = 1500, 4096
    W = [torch.from_numpy(rng.standard_normal((N, K))).half().cuda() for _ in range(3)]
    x, xh = codes(rng, M, K)
    xs, xsh = scales(rng, M)
    buf = torch.empty(N, K, dtype=torch.int8, device="cuda")
    s = torch.empty(N, device="cuda")
    want = []
    for w in W:
        q, qs = quantize_ref(w.double().cpu().numpy())
        want.append(torch.from_numpy(scaled_f32(product(xh, q), xsh, qs)).bfloat16())
    ys = []
    torch.cuda.synchronize()
    for i in range(60):
        m.wq_quantize_i8(W[i % 3], codes=buf, scales=s)
        ys.append(m.wq_gemm_i8(x, xs, buf, s))
    for i, y in enumerate(ys):
        assert torch.equal(y.cpu(), want[i % 3]), i


@pytest.mark.parametrize("M", [1, 16, 100, 300])
def test_outputs_overwritten_call_after_call(M):
    """Calls that write the same output, and read what the last one wrote, without a wait between."""
    m = wq()
    rng = np.random.default_rng([2, M])
    D = 640
    w = [m.wq_quantize_i8(torch.from_numpy(rng.standard_normal((D, D)) * 0.06).half().cuda()) for _ in range(3)]
    x0 = torch.from_numpy(rng.standard_normal((M, D))).bfloat16().cuda()

    def chain(wait):
        h = x0.clone()
        q, qs = torch.empty(M, D, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        for i in range(12):
            m.wq_quantize_i8(h, codes=q, scales=qs)
            if wait:
                torch.cuda.synchronize()
            if i % 3 == 2:
                m.wq_gated_i8(q, qs, *w[0], *w[1], h=h)
            else:
                m.wq_gemm_i8(q, qs, *w[i % 3], y=h)
            if wait:
                torch.cuda.synchronize()
        return h

    want = chain(True)
    assert torch.isfinite(want.float()).all()
    for _ in range(10):
        assert torch.equal(chain(False), want)


def test_beside_the_weight_only_calls():
    """A weight-only prefill product (two launches, the second a dependent one), its
    result quantised, an 8-bit block, and the weight-only product again: as with waits between."""
    m = wq()
    rng = np.random.default_rng(3)
    M, K, N = 2048, 1024, 5120
    W = torch.from_numpy(wq_inputs.weight_f16(3, 0, N, K)).cuda()
    c, s, z = m.wq_quantize_rtn(W, 4, 128)
    c2, s2, z2 = m.wq_quantize_rtn(torch.from_numpy(wq_inputs.weight_f16(3, 1, K, N)).cuda(), 4, 128)
    w8 = m.wq_quantize_i8(torch.from_numpy(0.02 * rng.standard_normal((N, N))).half().cuda())
    x = wq_inputs.activations_bf16(3, 2, M, K).cuda()

    def chain(wait):
        steps = []
        y = m.wq_gemm(x, c, s, z, 4, 128, N, K)
        for _ in range(3):
            if wait:
                torch.cuda.synchronize()
            q, qs = m.wq_quantize_i8(y)
            if wait:
                torch.cuda.synchronize()
            h = m.wq_gemm_i8(q, qs, *w8)
            if wait:
                torch.cuda.synchronize()
            back = m.wq_gemm(h, c2, s2, z2, 4, 128, K, N)
            y = m.wq_gemm(back, c, s, z, 4, 128, N, K)
            steps += [q, qs, h, back, y]
        return steps

    want = chain(True)
    for _ in range(3):
        for a, b in zip(chain(False), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_two_threads_two_streams(M):
    m = wq()
    rng = np.random.default_rng([4, M])
    N, K = 900, 1111
    w, _ = codes(rng, N, K)
    ws, _ = scales(rng, N)
    xs, _ = scales(rng, M)
    xx = [codes(rng, M, K)[0] for _ in range(2)]
    want = [m.wq_gemm_i8(x, xs, w, ws) for x in xx]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        st = torch.cuda.Stream()
        for _ in range(200):
            y = m.wq_gemm_i8(xx[i], xs, w, ws, stream=st)
            st.synchronize()
            if not torch.equal(y, want[i]):
                bad.append(i)
                return

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


@pytest.mark.parametrize("M", [1, 20, 300])
def test_weights_past_4_gib(M):
    """Rows of a weight matrix whose offsets pass 2^32 bytes."""
    m = wq()
    rng = np.random.default_rng([5, M])
    N, K = 35000, 131056
    w = torch.empty(N, K, dtype=torch.int8, device="cuda")
    w[:] = torch.randint(-127, 128, (1, K), dtype=torch.int8, device="cuda")
    part, ph = codes(rng, 200, K)
    w[-200:] = part
    x, xh = codes(rng, M, K)
    xs, xsh = scales(rng, M)
    ws, wsh = scales(rng, N)
    y = m.wq_gemm_i8(x, xs, w, ws, dtype=torch.float32)
    np.testing.assert_array_equal(y[:, -200:].cpu().numpy(), scaled_f32(product(xh, ph), xsh, wsh[-200:]))
    g = m.wq_gated_i8(x, xs, w[-300:], ws[-300:], w[:300], ws[:300])
    g2 = m.wq_gated_i8(x, xs, w[-300:].clone(), ws[-300:], w[:300].clone(), ws[:300])
    assert torch.equal(g, g2)


def test_results_past_2_to_32_elements():
    m = wq()
    rng = np.random.default_rng(6)
    M, N, K = 66000, 65600, 48
    w, wh = codes(rng, N, K)
    ws, wsh = scales(rng, N)
    x = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda")
    xs = torch.rand(M, device="cuda") + 0.5
    y = m.wq_gemm_i8(x, xs, w, ws)
    for rows in (slice(0, 130), slice(M - 130, M)):
        want = scaled_f32(product(x[rows].cpu().numpy(), wh), xs[rows].cpu().numpy(), wsh)
        assert torch.equal(y[rows].cpu(), torch.from_numpy(want).bfloat16())
    del y
    q, qs = m.wq_quantize_i8(torch.rand(34000, 130000, device="cuda", dtype=torch.bfloat16))
    last = slice(33990, 34000)
    x = torch.rand(10, 130000, device="cuda", dtype=torch.bfloat16)
    big = torch.zeros(34000, 130000, device="cuda", dtype=torch.bfloat16)
    big[last] = x
    m.wq_quantize_i8(big, codes=q, scales=qs)
    rq, rs = quantize_ref(x.double().cpu().numpy())
    np.testing.assert_array_equal(q[last].cpu().numpy(), rq)
    np.testing.assert_array_equal(qs[last].cpu().numpy(), rs)
    assert (qs[:33990] == 0).all() and not q[:33990:997].any()


def _first_call_child(q, M):
    import sys
    sys.path.insert(0, ROOT)
    try:
        import torch

        import quantized_gemm_wq_b200 as wq
        K, N = 512, 768
        x = torch.randn(M, K, device="cuda").bfloat16()
        w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
        ws = torch.rand(N, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):                     # the process's first calls are the captured ones
            c, s = wq.wq_quantize_i8(x)
            y = wq.wq_gemm_i8(c, s, w, ws)
            h = wq.wq_gated_i8(c, s, w, ws, w, ws)
        g.replay()
        torch.cuda.synchronize()
        c2, s2 = wq.wq_quantize_i8(x)
        q.put(bool(torch.equal(c, c2) and torch.equal(y, wq.wq_gemm_i8(c2, s2, w, ws))
                   and torch.equal(h, wq.wq_gated_i8(c2, s2, w, ws, w, ws))))
    except Exception as e:  # noqa: BLE001
        q.put(repr(e))


@pytest.mark.parametrize("M", [4, 40, 300])
def test_first_calls_may_be_captured(M):
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    pr = ctx.Process(target=_first_call_child, args=(q, M))
    pr.start()
    res = q.get(timeout=300)
    pr.join(60)
    assert res is True, res


@pytest.mark.parametrize("M", [1, 8, 100, 300])
def test_tokens_rewritten_just_before_the_product(M):
    """The same codes and scales buffers for other tokens at every step, with the products of
    the steps before still reading them: no step sees what an earlier one left in a cache."""
    m = wq()
    rng = np.random.default_rng([7, M])
    N, K = 2304, 512
    w, wh = codes(rng, N, K)
    ws, wsh = scales(rng, N)
    xs = [torch.from_numpy(rng.standard_normal((M, K))).bfloat16().cuda() for _ in range(5)]
    want = []
    for x in xs:
        q, qs = quantize_ref(x.double().cpu().numpy())
        want.append(torch.from_numpy(scaled_f32(product(q, wh), qs, wsh)).bfloat16().cuda())
    buf, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    ys = torch.empty(300, M, N, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):                         # back to back on the GPU
        for i in range(300):
            m.wq_quantize_i8(xs[i % 5], codes=buf, scales=s)
            m.wq_gemm_i8(buf, s, w, ws, y=ys[i])
    for _ in range(3):
        ys.zero_()
        g.replay()
        for i in range(300):
            assert torch.equal(ys[i], want[i % 5]), i


def _child(q):
    import sys
    sys.path.insert(0, ROOT)
    sys.path.insert(0, os.path.join(ROOT, "tests"))
    try:
        import numpy as np
        import torch

        import quantized_gemm_wq_b200 as wq
        short = ctypes.CDLL(os.path.join(ROOT, "quantized_gemm_wq_b200", "libwq_shortwait.so"))
        for name in ("wq_gemm_i8", "wq_gated_i8", "wq_last_device_error"):
            getattr(short, name).argtypes = getattr(wq.lib, name).argtypes
            getattr(short, name).restype = getattr(wq.lib, name).restype
        res = {}
        N, K = 640, 4096
        p = lambda t: t.data_ptr()
        w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
        ws = torch.rand(N, device="cuda")
        for M in (40, 128, 300):
            x = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda")
            xs = torch.rand(M, device="cuda")
            y = torch.empty(M, N, device="cuda")
            res[f"gemm {M}"] = short.wq_gemm_i8(p(x), K, p(xs), M, N, K, p(w), K, p(ws), p(y), 2, N, None)
            res[f"gemm {M} error"] = short.wq_last_device_error()
            res[f"gated {M}"] = short.wq_gated_i8(p(x), K, p(xs), M, N, K, p(w), p(ws), p(w), p(ws), K, 0, p(y), 2, N, None)
            res[f"gated {M} error"] = short.wq_last_device_error()
            res[f"cleared {M}"] = short.wq_last_device_error()
            got = wq.wq_gemm_i8(x, xs, w, ws, dtype=torch.float32).cpu().numpy()
            acc = x.cpu().numpy().astype(np.float64) @ w.cpu().numpy().astype(np.float64).T
            ref = (acc.astype(np.float32) * xs.cpu().numpy()[:, None]) * ws.cpu().numpy()[None, :]
            res[f"after {M}"] = bool(np.array_equal(got, ref))
            res[f"after {M} error"] = wq.wq_last_device_error()
        q.put(res)
    except Exception as e:  # noqa: BLE001
        q.put({"exception": repr(e)})


def test_waits_that_run_out():
    """The test build whose pipeline waits have no time: each wait of the tensor-core
    kernels finds its barrier complete or is given up, the copies and MMAs in flight
    are seen out, an error is reported at most once, and right after the library proper
    computes right results in the same context."""
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    pr = ctx.Process(target=_child, args=(q,))
    pr.start()
    res = q.get(timeout=300)
    pr.join(60)
    assert "exception" not in res, res
    for M in (40, 128, 300):
        assert res[f"gemm {M}"] == 0 and res[f"gated {M}"] == 0
        assert res[f"gemm {M} error"] in (0, 8) and res[f"gated {M} error"] in (0, 8)   # done, or gave up
        assert res[f"cleared {M}"] == 0
        assert res[f"after {M}"] is True and res[f"after {M} error"] == 0
