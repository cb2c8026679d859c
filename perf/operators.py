"""Cases of the 8-bit integer linear operators: wq_quantize_i8, wq_gemm_i8, wq_gated_i8.

Both sides of a linear layer are 8-bit integers here: the activations with one
scale for each token (taken from the token's own largest value at run time),
the weights with one scale for each output channel.  With a row x of length K,

    s = fp32(max|x| / 127)      q = round_half_even(x / s), 0 where s = 0
    y[m, n] = s_x[m] s_w[n] sum_k q_x[m, k] q_w[n, k]
    h[m, n] = act(g[m, n]) u[m, n],  g and u as y with the gate's and the up projection's weights

A case's "op" is one of these calls, or "block": a whole gated feed-forward
block, quantise -> gated -> quantise -> product, as a model layer runs it.
"""
import math

import torch

own = False   # set by the program that measures: True makes the calls of this repository's package

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one token's hidden state before a projection: the smallest call, all latency
        {"name": "quantize one token", "op": "quantize", "M": 1, "K": 4096, "type": "bf16", "pad": 0},
        # the product of a gated block over a prompt of 2048 tokens, before its down projection
        {"name": "quantize prompt", "op": "quantize", "M": 2048, "K": 13824, "type": "bf16", "pad": 0},
        # a projection's weights, once at load time
        {"name": "quantize weights", "op": "quantize", "M": 13824, "K": 5120, "type": "f16", "pad": 0},
        # a ragged batch of fp32 activations that are columns of a wider buffer
        {"name": "quantize ragged view", "op": "quantize", "M": 777, "K": 5003, "type": "f32", "pad": 29},
        # decode, one request: an attention projection
        {"name": "gemm one token", "op": "gemm", "M": 1, "N": 4096, "K": 4096, "type": "bf16", "pad": 0},
        # decode, sixteen requests: the widest projection of the benchmark's shapes, 604 MB of weights
        {"name": "gemm 16 tokens", "op": "gemm", "M": 16, "N": 49152, "K": 12288, "type": "bf16", "pad": 0},
        # decode, a batch of 64: an up projection
        {"name": "gemm 64 tokens", "op": "gemm", "M": 64, "N": 11008, "K": 4096, "type": "bf16", "pad": 0},
        # prefill of 2048 tokens: a down projection, long sums
        {"name": "gemm prompt", "op": "gemm", "M": 2048, "N": 5120, "K": 13824, "type": "bf16", "pad": 0},
        # a ragged prompt, odd sizes, rows inside wider buffers, fp32 result (logits)
        {"name": "gemm ragged view", "op": "gemm", "M": 333, "N": 4999, "K": 5003, "type": "f32", "pad": 48},
        # decode, one request: gate and up projections of a block
        {"name": "gated one token", "op": "gated", "M": 1, "N": 11008, "K": 4096, "type": "bf16", "pad": 0, "act": "silu"},
        # prefill of 2048 tokens: gate and up projections of a block
        {"name": "gated prompt", "op": "gated", "M": 2048, "N": 13824, "K": 5120, "type": "bf16", "pad": 0, "act": "silu"},
        # decode, eight requests: the whole feed-forward block, four calls in a row
        {"name": "block 8 tokens", "op": "block", "M": 8, "N": 11008, "K": 4096, "type": "bf16", "pad": 0, "act": "silu"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "gemm", "gemm", "gated", "gated", "block"))
    case = {"op": op, "M": _log(rng, 1, 2048), "K": _log(rng, 64, 13824)}
    if op != "quantize":
        case["N"] = _log(rng, 64, 13824)
    if rng.random() < 0.5:      # half of the sizes are multiples of 64, as models have them, half are whatever comes
        for k in ("N", "K"):
            if k in case:
                case[k] = 64 * max(1, case[k] // 64)
    case["type"] = rng.choice(("bf16", "bf16", "f16", "f32"))
    case["pad"] = rng.choice((0, 0, 16, 80))
    if op in ("gated", "block"):
        case["act"] = rng.choice(("silu", "gelu", "gelu_tanh"))
    most = 2 * 2048 * 13824 * 5120      # multiply-adds of the largest listed case
    parts = {"quantize": 0, "gemm": 1, "gated": 2, "block": 3}[op]
    if parts:
        case["M"] = max(1, min(case["M"], most // (parts * case["N"] * case["K"])))
    return case


# ---------------------------------------------------------------- inputs

def _round(x, s):
    """Codes of the values x on the grids s (one a row)."""
    s = s[:, None].double()
    return torch.where(s > 0, torch.round(x.double() / torch.where(s > 0, s, 1.0)), 0.0).clamp_(-127, 127).to(torch.int8)


def _activations(gen, M, K):
    """Hidden states: unit normal, one feature in fifty 20 times as large, rows of different size; the last of several rows
    is a padded token, all zero."""
    x = torch.randn(M, K, device="cuda", generator=gen)
    x *= torch.where(torch.rand(K, device="cuda", generator=gen) < 0.02, 20.0, 1.0)
    x *= torch.exp(0.5 * torch.randn(M, 1, device="cuda", generator=gen))
    if M > 2:
        x[M - 1] = 0.0
    return x


def _in_buffer(x, pad, align):
    """x as the first columns of a wider buffer, whose other columns hold values that no result may depend on."""
    M, K = x.shape
    ld = -(-K // align) * align + pad
    if ld == K:
        return x.contiguous()
    wide = torch.full((M, ld), 77, dtype=x.dtype, device=x.device)
    wide[:, :K] = x
    return wide[:, :K]


def _weights(gen, N, K, pad):
    """Codes and scales of normal weights, 4096 rows at a time."""
    ld = -(-K // 16) * 16 + pad
    codes = torch.full((N, ld), 77, dtype=torch.int8, device="cuda")[:, :K]
    scales = torch.empty(N, device="cuda")
    for n in range(0, N, 4096):
        w = (0.02 * torch.randn(min(4096, N - n), K, device="cuda", generator=gen)).half().float()
        s = w.abs().amax(1) / 127
        scales[n:n + 4096] = s
        codes[n:n + 4096] = torch.clamp(torch.round(w / s[:, None]), -127, 127).to(torch.int8)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, M, K, pad = case["op"], case["M"], case["K"], case["pad"]
    state = {"op": op, "type": _TYPES[case["type"]], "act": case.get("act")}
    x = _activations(gen, M, K)
    if op in ("quantize", "block"):
        # a row may start anywhere in a wider buffer when it is quantised; "pad" counts elements of its type
        state["x"] = _in_buffer(x.to(_TYPES[case["type"]]), pad, 1)
    else:
        s = x.abs().amax(1) / 127
        state["x"], state["xs"] = _in_buffer(_round(x, s), pad, 16), s
    if op == "gemm":
        state["w"], state["ws"] = _weights(gen, case["N"], K, pad)
    if op in ("gated", "block"):
        state["wg"], state["gs"] = _weights(gen, case["N"], K, pad)
        state["wu"], state["us"] = _weights(gen, case["N"], K, pad)
    if op == "block":
        state["wd"], state["ds"] = _weights(gen, K, case["N"], pad)
    return state


# ---------------------------------------------------------------- one pass

def _plain_quantize(x):
    s = x.float().abs().amax(1) / 127
    return _round(x, s), s          # the quotients in 64 bits: a code next to a half is decided by the exact one


def _plain_product(x, xs, w, ws):
    return x.float() @ w.float().t() * xs[:, None] * ws[None, :]


def _plain_act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * torch.erfc(-g * math.sqrt(0.5))
    return g / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain_gated(x, xs, s):
    return _plain_act(_plain_product(x, xs, s["wg"], s["gs"]), s["act"]) * _plain_product(x, xs, s["wu"], s["us"])


def run(s):
    op = s["op"]
    if own:
        import quantized_gemm_wq_b200 as wq
        if op == "quantize":
            codes, scales = wq.wq_quantize_i8(s["x"])
            return {"codes": codes, "scales": scales}
        if op == "gemm":
            return wq.wq_gemm_i8(s["x"], s["xs"], s["w"], s["ws"], dtype=s["type"])
        if op == "gated":
            return wq.wq_gated_i8(s["x"], s["xs"], s["wg"], s["gs"], s["wu"], s["us"], act=s["act"], dtype=s["type"])
        q, qs = wq.wq_quantize_i8(s["x"])
        h = wq.wq_gated_i8(q, qs, s["wg"], s["gs"], s["wu"], s["us"], act=s["act"], dtype=s["type"])
        q, qs = wq.wq_quantize_i8(h)
        return {"h": h, "y": wq.wq_gemm_i8(q, qs, s["wd"], s["ds"], dtype=s["type"])}
    if op == "quantize":
        codes, scales = _plain_quantize(s["x"])
        return {"codes": codes, "scales": scales}     # codes are whole numbers; codes times scales are the values they stand for
    if op == "gemm":
        return _plain_product(s["x"], s["xs"], s["w"], s["ws"]).to(s["type"])
    if op == "gated":
        return _plain_gated(s["x"], s["xs"], s).to(s["type"])
    q, qs = _plain_quantize(s["x"])
    h = _plain_gated(q, qs, s).to(s["type"])
    q, qs = _plain_quantize(h)
    return {"h": h, "y": _plain_product(q, qs, s["wd"], s["ds"]).to(s["type"])}


def work(case):
    op, M, K, N = case["op"], case["M"], case["K"], case.get("N", 0)
    e = _BYTES[case["type"]]
    if op == "quantize":
        return {"bytes": M * K * (e + 1) + 4 * M, "flops": 3 * M * K}
    if op == "gemm":
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * e, "flops": 2 * M * N * K}
    if op == "gated":
        return {"bytes": M * K + 2 * N * K + 4 * (M + 2 * N) + M * N * e, "flops": 4 * M * N * K}
    return {"bytes": M * K * e + 3 * N * K + 4 * (2 * N + K) + M * (N + K) * e, "flops": 6 * M * N * K}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_linear(q, qs, w, ws):
    """sum over k of (q s)(w t) for every pair of rows, in blocks of 2048 rows of w."""
    a = q.to(torch.float64) * qs.double().unsqueeze(1)
    parts = [torch.matmul(a, (w[n:n + 2048].to(torch.float64) * ws[n:n + 2048].double().unsqueeze(1)).transpose(0, 1))
             for n in range(0, w.shape[0], 2048)]
    return torch.cat(parts, dim=1)


def _exact_act(g, act):
    if act == "silu":
        return g * torch.special.expit(g)
    if act == "gelu":
        return g * torch.special.ndtr(g)
    return g * (0.5 + 0.5 * torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        return {"codes": None, "scales": s["x"].double().abs().amax(dim=1) / 127.0}
    if s["op"] == "gemm":
        return _exact_linear(s["x"], s["xs"], s["w"], s["ws"])

    def gated(q, qs):
        return _exact_act(_exact_linear(q, qs, s["wg"], s["gs"]), s["act"]) * _exact_linear(q, qs, s["wu"], s["us"])

    def codes(v):       # the scale is held in 32 bits; the quotient is taken in 64
        t = (v.double().abs().amax(dim=1) / 127.0).float()
        q = torch.round(v.double() / t.double().unsqueeze(1))
        return torch.nan_to_num(q, nan=0.0), t

    if s["op"] == "gated":
        return gated(s["x"], s["xs"])
    h = gated(*codes(s["x"]))
    return {"h": h, "y": _exact_linear(*codes(h.to(s["type"])), s["wd"], s["ds"])}
