"""wq_quantize_i8, wq_gemm_i8 and wq_gated_i8 on the GPU against their
definition in 64 bits: codes, scales and products bit for bit, the gated call
within the roundings that its formula has."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from i8_util import assert_rounds_to, codes, gated_ref, product, quantize_ref, scaled_f32, scales, wq

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
CANARY = 0x5A


def _rows(rng, R, K, dtype):
    x = rng.standard_normal((R, K)) * np.exp(rng.normal(0, 1, (R, 1)))
    x[:, rng.random(K) < 0.02] *= 20
    return torch.from_numpy(x).to(dtype)


def _check_quantize(x_dev, x_host):
    q, s = wq().wq_quantize_i8(x_dev)
    rq, rs = quantize_ref(x_host.double().numpy())
    assert q.dtype == torch.int8 and s.dtype == torch.float32 and q.shape == x_host.shape
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


# ------------------------------------------------------------------ quantise

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,K", [(1, 1), (1, 7), (3, 8), (5, 31), (2, 257), (9, 512), (17, 1000), (1, 4096),
                                 (33, 5003), (4, 16384), (3, 16385), (2, 40000), (1, 131071)])
def test_quantize(R, K, dtype):
    rng = np.random.default_rng([R, K])
    x = _rows(rng, R, K, dtype)
    _check_quantize(x.cuda(), x)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [1, 3, 5, 8])
@pytest.mark.parametrize("K,ld", [(5, 21), (200, 213), (4099, 4111), (17000, 17011)])
def test_quantize_rows_start_anywhere(dtype, shift, K, ld):
    """Rows inside a wider buffer, at element offsets that are no multiple of 16 bytes."""
    rng = np.random.default_rng(K)
    wide = _rows(rng, 6, ld + 8, dtype)
    _check_quantize(wide.cuda()[:, shift:shift + K], wide[:, shift:shift + K])


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_halves(dtype):
    """Every quotient exactly on a half, or one step of the type beside it:
    scales that are powers of two, and scales that are not."""
    rows = []
    for e in (0, -3, 5):
        half = (np.arange(254) - 127 + 0.5) * 2.0 ** e
        t = torch.from_numpy(half).to(dtype)
        up = torch.nextafter(t, torch.tensor(float("inf"), dtype=dtype))
        dn = torch.nextafter(t, torch.tensor(float("-inf"), dtype=dtype))
        rows.append(torch.cat([t, up, dn, torch.tensor([127.0 * 2.0 ** e]).to(dtype)]))
    x = torch.stack(rows)
    _check_quantize(x.cuda(), x)
    rng = np.random.default_rng(1)
    # maxima whose scale has a full significand, and values nearest to its halves
    a = torch.from_numpy(rng.uniform(0.5, 2.0, (64, 1))).to(dtype).double()
    s = (a / 127.0).float().double()
    near = ((torch.arange(126).double() + 0.5)[None] * s).to(dtype)
    x = torch.cat([near, torch.nextafter(near, torch.full_like(near, 9.0)), torch.nextafter(near, torch.zeros_like(near)),
                   a.to(dtype)], 1)
    _check_quantize(x.cuda(), x)
    _check_quantize(-x.cuda(), -x)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_extremes(dtype):
    """Rows of zeros, of the smallest and the largest values, of signed zeros, of non-finite values."""
    f = torch.finfo(dtype)
    tiny = f.smallest_normal * f.eps        # the smallest subnormal
    rng = np.random.default_rng(2)
    base = torch.from_numpy(rng.uniform(-1, 1, (12, 100)))
    x = torch.zeros(12, 100, dtype=torch.float64)
    x[1] = -0.0
    x[2] = torch.round(base[2] * 3) * tiny
    x[3] = torch.round(base[3] * 300) * tiny
    x[4] = base[4] * f.smallest_normal * 200
    x[5] = base[5] * f.max
    x[5, 7] = f.max
    x[6] = base[6]
    x[6, 99] = float("inf")
    x[7, 3] = float("-inf")
    x[8] = base[8]
    x[8, 0] = float("nan")
    x[9, 50] = float("nan")
    x[9, 51] = float("inf")
    x[10, 98] = tiny
    x[11] = base[11] * (2.0 ** -95 if dtype != torch.float16 else 1.0)
    x = x.to(dtype)
    _check_quantize(x.cuda(), x)


def test_quantize_writes_its_rows_only():
    rng = np.random.default_rng(3)
    x = _rows(rng, 5, 100, torch.bfloat16).cuda()
    wide = torch.full((7, 160), CANARY, dtype=torch.int8, device="cuda")
    s = torch.full((7,), 7.0, device="cuda")
    q, qs = wq().wq_quantize_i8(x, codes=wide[1:6, 16:116], scales=s[1:6])
    rq, rs = quantize_ref(x.double().cpu().numpy())
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(qs.cpu().numpy(), rs)
    w = wide.cpu().numpy()
    assert (w[0] == CANARY).all() and (w[6] == CANARY).all() and (w[:, :16] == CANARY).all() and (w[:, 116:] == CANARY).all()
    assert s[0] == 7.0 and s[6] == 7.0


# ------------------------------------------------------------------ product

SHAPES = [(1, 1, 1), (1, 5, 17), (1, 16, 64), (1, 33, 4096), (2, 100, 63), (3, 128, 65), (7, 129, 1000), (8, 48, 256),
          (9, 200, 511), (15, 77, 513), (16, 256, 2048), (17, 130, 300), (31, 64, 128), (32, 300, 1024), (33, 257, 130),
          (64, 384, 4096), (65, 96, 777), (100, 1000, 1500), (128, 512, 512), (129, 140, 384), (200, 333, 5003),
          (255, 256, 640), (256, 1024, 2048), (257, 129, 200), (300, 700, 1111), (512, 512, 4096), (513, 1030, 260),
          (1025, 260, 400)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K):
    rng = np.random.default_rng([M, N, K])
    x, xh = codes(rng, M, K)
    w, wh = codes(rng, N, K)
    xs, xsh = scales(rng, M)
    ws, wsh = scales(rng, N)
    ref = scaled_f32(product(xh, wh), xsh, wsh)
    y = wq().wq_gemm_i8(x, xs, w, ws, dtype=torch.float32)
    np.testing.assert_array_equal(y.cpu().numpy(), ref)
    for dtype in (torch.bfloat16, torch.float16):
        y = wq().wq_gemm_i8(x, xs, w, ws, dtype=dtype)
        assert y.dtype == dtype
        torch.testing.assert_close(y.cpu(), torch.from_numpy(ref).to(dtype), rtol=0, atol=0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K,pad,ypad", [(1, 40, 100, 16, 3), (5, 61, 90, 32, 1), (16, 130, 513, 16, 7),
                                            (40, 97, 200, 48, 5), (130, 250, 333, 16, 8), (300, 513, 257, 80, 11)])
def test_gemm_views(M, N, K, pad, ypad, dtype):
    """Operands and result inside wider buffers; what lies around the result stays."""
    rng = np.random.default_rng([M, N, K, 1])
    x, xh = codes(rng, M, K, pad)
    w, wh = codes(rng, N, K, pad + 16)
    xs, xsh = scales(rng, M)
    ws, wsh = scales(rng, N)
    wide = torch.full((M + 2, N + ypad + 2), 7.0, dtype=dtype, device="cuda")
    y = wq().wq_gemm_i8(x, xs, w, ws, y=wide[1:M + 1, 1:N + 1])
    ref = torch.from_numpy(scaled_f32(product(xh, wh), xsh, wsh)).to(dtype)
    torch.testing.assert_close(y.cpu(), ref, rtol=0, atol=0)
    wide[1:M + 1, 1:N + 1] = 7.0
    assert (wide == 7.0).all()


@pytest.mark.parametrize("M", [1, 12, 40, 300])
def test_gemm_largest_sums(M):
    """The longest row with the largest codes: sums of 2^14 (2^17 - 1), one step from int32's end."""
    K, N = 131071, 130
    x = torch.full((M, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
    w = torch.full((N, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
    w[1] = 127
    w[2, ::2] = 127
    one = torch.ones(max(M, N), device="cuda")
    y = wq().wq_gemm_i8(x, one[:M], w, one[:N], dtype=torch.float32)
    acc = [2 ** 14 * K, -128 * 127 * K, 2 ** 14 * (K // 2) - 128 * 127 * (K // 2 + 1)]
    want = torch.tensor([float(np.float32(a)) for a in acc])
    assert (y[:, :3].cpu() == want).all() and (y[:, 3:] == float(np.float32(acc[0]))).all()


@pytest.mark.parametrize("M", [1, 20, 300])
def test_gemm_scales_that_leave_the_range(M):
    """Zero, subnormal, huge, infinite and NaN scales, each in its own row or column."""
    rng = np.random.default_rng(5)
    N, K = 70, 200
    x, xh = codes(rng, M, K)
    w, wh = codes(rng, N, K)
    xs, xsh = scales(rng, M)
    ws, wsh = scales(rng, N)
    for i, v in enumerate((0.0, 1e-42, 1e38, np.inf, np.nan)):
        wsh[3 * i] = v
        if 2 * i < M:
            xsh[2 * i] = v
    ws.copy_(torch.from_numpy(wsh))
    xs.copy_(torch.from_numpy(xsh))
    y = wq().wq_gemm_i8(x, xs, w, ws, dtype=torch.float32)
    np.testing.assert_array_equal(y.cpu().numpy(), scaled_f32(product(xh, wh), xsh, wsh))


@pytest.mark.parametrize("call", ["gemm", "gated"])
def test_rows_do_not_depend_on_the_batch(call):
    """The same tokens, alone and in batches that other kernels take: the same bits."""
    rng = np.random.default_rng(6)
    N, K = 260, 700
    x, _ = codes(rng, 600, K)
    xs, _ = scales(rng, 600)
    w, _ = codes(rng, N, K)
    ws, _ = scales(rng, N)
    u, _ = codes(rng, N, K)
    us, _ = scales(rng, N)

    def run(rows):
        if call == "gemm":
            return wq().wq_gemm_i8(x[rows], xs[rows], w, ws)
        return wq().wq_gated_i8(x[rows], xs[rows], w, ws, u, us)

    full = run(slice(0, 600))
    for m in (1, 2, 8, 9, 16, 17, 40, 130, 257):
        assert torch.equal(run(slice(5, 5 + m)), full[5:5 + m]), m


# ------------------------------------------------------------------ gated

@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 30, 100), (1, 257, 4096), (4, 64, 65), (8, 100, 640), (9, 33, 129),
                                   (16, 130, 1000), (33, 70, 300), (64, 256, 2048), (127, 65, 257), (130, 200, 500),
                                   (256, 129, 1024), (260, 300, 400), (520, 513, 1024)])
def test_gated(M, N, K, act):
    rng = np.random.default_rng([M, N, K, 2])
    x, xh = codes(rng, M, K)
    g, gh = codes(rng, N, K)
    u, uh = codes(rng, N, K, 0)
    xs, xsh = scales(rng, M)
    gs, gsh = scales(rng, N)
    us, ush = scales(rng, N)
    # gate values over the activation's whole range: unit size times the scales' spread
    gs *= 1.0 / (74.0 ** 2 * K ** 0.5 * 1e-3)
    gsh = gs.cpu().numpy()
    ref, err = gated_ref(product(xh, gh), product(xh, uh), xsh, gsh, ush, act)
    for dtype in TYPES:
        h = wq().wq_gated_i8(x, xs, g, gs, u, us, act=act, dtype=dtype)
        assert h.dtype == dtype and h.shape == (M, N)
        assert_rounds_to(h, ref, err,
                         f"{act} {dtype}")


@pytest.mark.parametrize("M,N,K,pad,hpad", [(1, 40, 100, 16, 3), (12, 61, 90, 32, 1), (50, 130, 513, 16, 7),
                                            (300, 250, 333, 16, 8)])
def test_gated_views(M, N, K, pad, hpad):
    rng = np.random.default_rng([M, N, K, 3])
    x, _ = codes(rng, M, K, pad)
    g, _ = codes(rng, N, K, pad)
    u, _ = codes(rng, N, K, pad)
    xs, _ = scales(rng, M)
    gs, _ = scales(rng, N)
    us, _ = scales(rng, N)
    wide = torch.full((M + 2, N + hpad + 2), 7.0, dtype=torch.bfloat16, device="cuda")
    h = wq().wq_gated_i8(x, xs, g, gs, u, us, h=wide[1:M + 1, 1:N + 1])
    want = wq().wq_gated_i8(*[t.clone() if t.dim() == 1 else _repack(t) for t in (x, xs, g, gs, u, us)])
    assert torch.equal(h, want)
    wide[1:M + 1, 1:N + 1] = 7.0
    assert (wide == 7.0).all()


def _repack(t):
    ld = (t.shape[1] + 15) // 16 * 16
    wide = torch.zeros(t.shape[0], ld, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_activations_over_their_range(M, act):
    """g on a fine grid (the gate's scales carry it), u = 1: the activation itself, fp32."""
    g = np.concatenate([np.linspace(-13, 13, 20001), np.linspace(-1, 1, 4001), np.linspace(-120, 120, 4001),
                        [0.0, -0.0, 1e-30, -1e-30, 1e-40, 3e4, -3e4]]).astype(np.float32)
    N = len(g)
    x = torch.zeros(M, 16, dtype=torch.int8, device="cuda")
    x[:, 0] = 1
    w = torch.zeros(N, 16, dtype=torch.int8, device="cuda")
    w[:, 0] = 1
    h = wq().wq_gated_i8(x, torch.ones(M, device="cuda"), w, torch.from_numpy(g).cuda(), w,
                         torch.ones(N, device="cuda"), act=act, dtype=torch.float32)
    one = np.ones((1, N))
    ref, err = gated_ref(one, one, np.ones(1, np.float32), g, np.ones(N, np.float32), act)
    assert_rounds_to(h[:1], ref, err, act)
    assert torch.equal(h, h[:1].expand(M, N))


def test_gated_zero_gate_and_saturated_gate():
    """g = 0 gives 0; a gate far below zero gives (a signed) 0, far above g u."""
    K, N = 64, 48
    x = torch.ones(3, K, dtype=torch.int8, device="cuda")
    g = torch.ones(N, K, dtype=torch.int8, device="cuda")
    u = torch.ones(N, K, dtype=torch.int8, device="cuda")
    one = torch.ones(N, device="cuda")
    xs = one[:3]
    gs = torch.zeros(N, device="cuda")
    gs[16:32] = -3.0       # g = -192
    gs[32:] = 3.0          # g = 192
    for act in ("silu", "gelu", "gelu_tanh"):
        h = wq().wq_gated_i8(x, xs, g, gs, u, one, act=act, dtype=torch.float32)
        assert (h[:, :32].abs() < 1e-30).all() and not torch.isnan(h).any(), act
        assert (h[:, 32:] == 192.0 * 64.0).all(), act


# ------------------------------------------------------------------ together

def _block(x, wg, wu, wd, dtype):
    m = wq()
    q, qs = m.wq_quantize_i8(x)
    h = m.wq_gated_i8(q, qs, *wg, *wu, dtype=dtype)
    q2, q2s = m.wq_quantize_i8(h)
    return q, qs, h, q2, q2s, m.wq_gemm_i8(q2, q2s, *wd, dtype=dtype)


@pytest.mark.parametrize("M,D,F", [(1, 256, 688), (6, 320, 500), (40, 130, 333), (150, 512, 1376), (400, 200, 700)])
@pytest.mark.parametrize("dtype", TYPES)
def test_feed_forward_block(M, D, F, dtype):
    """quantise -> gated -> quantise -> product, each step against its definition on what it was given."""
    rng = np.random.default_rng([M, D, F])
    m = wq()
    x = _rows(rng, M, D, dtype).cuda()
    w = [m.wq_quantize_i8(torch.from_numpy(0.05 * rng.standard_normal(s)).half().cuda())
         for s in ((F, D), (F, D), (D, F))]
    q, qs, h, q2, q2s, y = _block(x, *w, dtype)
    n = lambda t: t.cpu().numpy()
    rq, rs = quantize_ref(n(x.double()))
    np.testing.assert_array_equal(n(q), rq)
    np.testing.assert_array_equal(n(qs), rs)
    ref, err = gated_ref(product(rq, n(w[0][0])), product(rq, n(w[1][0])), rs, n(w[0][1]), n(w[1][1]), "silu")
    assert_rounds_to(h, ref, err)
    rq2, rs2 = quantize_ref(n(h.double()))
    np.testing.assert_array_equal(n(q2), rq2)
    np.testing.assert_array_equal(n(q2s), rs2)
    want = torch.from_numpy(scaled_f32(product(rq2, n(w[2][0])), rs2, n(w[2][1]))).to(dtype)
    torch.testing.assert_close(y.cpu(), want, rtol=0, atol=0)


def test_nan_token_stays_in_its_row():
    rng = np.random.default_rng(8)
    x = _rows(rng, 5, 128, torch.bfloat16).cuda()
    clean = x.clone()
    x[2, 17] = float("nan")
    w = [wq().wq_quantize_i8(_rows(rng, n, k, torch.float16).cuda()) for n, k in ((96, 128), (96, 128), (128, 96))]
    y = _block(x, *w, torch.bfloat16)[-1]
    want = _block(clean, *w, torch.bfloat16)[-1]
    assert torch.isnan(y[2]).all()
    keep = [0, 1, 3, 4]
    assert torch.equal(y[keep], want[keep])


@pytest.mark.parametrize("M", [1, 12, 64, 300])
def test_captured_and_replayed(M):
    """The block captured into a graph, replayed on new inputs, on two streams' graphs in turn."""
    rng = np.random.default_rng([9, M])
    w = [wq().wq_quantize_i8(_rows(rng, n, k, torch.float16).cuda()) for n, k in ((500, 256), (500, 256), (256, 500))]
    xin = _rows(rng, M, 256, torch.bfloat16).cuda()
    _block(xin, *w, torch.bfloat16)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _block(xin, *w, torch.bfloat16)[-1]
        graphs.append((g, out))
    for k in range(4):
        new = _rows(rng, M, 256, torch.bfloat16).cuda()
        want = _block(new, *w, torch.bfloat16)[-1]
        xin.copy_(new)
        g, out = graphs[k % 2]
        g.replay()
        assert torch.equal(out, want)


@pytest.mark.parametrize("M", [1, 16, 64, 300])
def test_runs_on_the_given_stream(M):
    """Work given to a stream waits for what that stream holds, and two calls at once do not disturb each other."""
    rng = np.random.default_rng([10, M])
    N, K = 700, 1024
    w, _ = codes(rng, N, K)
    ws, _ = scales(rng, N)
    xs, _ = scales(rng, M)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    xa, xb = (codes(rng, M, K)[0] for _ in range(2))
    want = [wq().wq_gemm_i8(t, xs, w, ws) for t in (xa, xb)]
    src = torch.zeros_like(xa)
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(a):
            torch.cuda._sleep(200000)
            src.copy_(xa)
        ya = wq().wq_gemm_i8(src, xs, w, ws, stream=a)
        yb = wq().wq_gemm_i8(xb, xs, w, ws, stream=b)
        torch.cuda.synchronize()
        assert torch.equal(ya, want[0]) and torch.equal(yb, want[1])
        src.zero_()
        torch.cuda.synchronize()


@pytest.mark.parametrize("M", [1, 12, 64, 300])
def test_failing_calls_write_nothing(M):
    m = wq()
    N, K = 256, 512
    rng = np.random.default_rng(11)
    x, _ = codes(rng, M, K)
    w, _ = codes(rng, N, K)
    xs, _ = scales(rng, M)
    ws, _ = scales(rng, N)
    y = torch.full((M, N), 7.0, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    L = m.lib
    assert L.wq_gemm_i8(p(x), K, p(xs), M, N, K, p(w), K, p(ws), p(y), 5, N, None) == m.WQ_ERR_TYPE
    assert L.wq_gemm_i8(p(x), K, p(xs), M, N, K, p(w), K, p(ws), p(y), 2, N - 1, None) == m.WQ_ERR_STRIDE
    assert L.wq_gemm_i8(p(x), K + 8, p(xs), M, N, K, p(w), K, p(ws), p(y), 2, N, None) == m.WQ_ERR_STRIDE
    assert L.wq_gemm_i8(p(x), K, p(xs), M, N, 0, p(w), K, p(ws), p(y), 2, N, None) == m.WQ_ERR_SHAPE
    assert L.wq_gated_i8(p(x), K, p(xs), M, N, K, p(w), p(ws), p(w), p(ws), K, 9, p(y), 2, N, None) == m.WQ_ERR_TYPE
    assert L.wq_gated_i8(p(x), K, p(xs), M, N, K, p(w), p(ws), None, p(ws), K, 0, p(y), 2, N, None) == m.WQ_ERR_NULL
    with pytest.raises(m.WQError):
        m.wq_gemm_i8(x[:0], xs[:0], w, ws)                  # no rows
    with pytest.raises(m.WQError):
        m.wq_gemm_i8(x[:, 8:], xs, w[:, 8:], ws, y=y)       # codes that start off a 16-byte boundary
    with pytest.raises(ValueError):
        m.wq_gemm_i8(x, xs, w[:, :500], ws, y=y)            # another K
    with pytest.raises(ValueError):
        m.wq_gemm_i8(x, xs.double(), w, ws, y=y)
    with pytest.raises(ValueError):
        m.wq_gemm_i8(x, xs, w, ws[:-1], y=y)
    with pytest.raises(ValueError):
        m.wq_gemm_i8(x, xs, w, ws, y=y[:, :-1])
    torch.cuda.synchronize()
    assert (y == 7.0).all()
    assert m.wq_last_device_error() == m.WQ_OK
