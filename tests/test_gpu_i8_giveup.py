"""The tensor-core kernels of the 8-bit integer linears when a bounded wait runs out.

The test build's hook makes one chosen wait of one CTA give up at once (the others
have 20 ms); copies and MMAs still complete.  In a child process: the call reports
the timeout exactly once, what it has stored are right results or nothing, and right
after, in the same context, the library proper computes right results."""
from __future__ import annotations

import ctypes
import multiprocessing as mp
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

EMPTY, FULL, DONE, ACC_EMPTY = range(4)
# name: (gated, M, N, K): 148 tiles unsplit; few tiles over clusters along K
SPLIT = {"unsplit": (False, 100, 18944, 4096), "unsplit gated": (True, 100, 9472, 4096),
         "clusters": (False, 40, 640, 32768), "clusters gated": (True, 40, 320, 32768)}
# (wait, cluster, rank, waits of its kind before it); every case has over 20 stages, fewer than 20 slots
SPLIT_WAITS = [(EMPTY, 2, 0, 20), (FULL, 2, 0, 0), (FULL, 2, 0, 20), (DONE, 2, 0, 0)]
CLUSTER_WAITS = [(EMPTY, 2, 1, 20), (FULL, 2, 1, 0), (FULL, 2, 1, 31), (DONE, 2, 1, 0)]


def _child(q, cases):
    import sys
    sys.path.insert(0, ROOT)
    try:
        import torch

        import quantized_gemm_wq_b200 as wq
        short = ctypes.CDLL(os.path.join(ROOT, "quantized_gemm_wq_b200", "libwq_shortwait.so"))
        for name in ("wq_gemm_i8", "wq_gated_i8", "wq_last_device_error"):
            getattr(short, name).argtypes = getattr(wq.lib, name).argtypes
            getattr(short, name).restype = getattr(wq.lib, name).restype
        out = []
        last = None
        p = lambda t: t.data_ptr()
        for (gated, M, N, K), wait in cases:
            if last != (gated, M, N, K):
                last = (gated, M, N, K)
                x = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda")
                w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
                u = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
                xs, ws = torch.rand(M, device="cuda"), torch.rand(N, device="cuda") * 1e-4
                call = (lambda: wq.wq_gated_i8(x, xs, w, ws, u, ws, dtype=torch.float32)) if gated else (
                    lambda: wq.wq_gemm_i8(x, xs, w, ws, dtype=torch.float32))
                want = call()
                assert torch.isfinite(want).all() and wq.wq_last_device_error() == 0
            y = torch.full((M, N), float("nan"), device="cuda")
            assert short.wq_test_give_up_i8(*wait) == 0
            if gated:
                st = short.wq_gated_i8(p(x), K, p(xs), M, N, K, p(w), p(ws), p(u), p(ws), K, 0, p(y), 2, N, None)
            else:
                st = short.wq_gemm_i8(p(x), K, p(xs), M, N, K, p(w), K, p(ws), p(y), 2, N, None)
            res = {"call": st, "error": short.wq_last_device_error(), "then": short.wq_last_device_error()}
            missing = torch.isnan(y)
            res["wrong"] = int((~missing & (y != want)).sum())
            rows, cols = missing.any(1).nonzero().flatten(), missing.any(0).nonzero().flatten()
            res["missing"] = int(missing.sum())
            res["rows"], res["cols"] = rows.numel(), cols.numel()
            res["first col"] = int(cols[0]) if cols.numel() else -1
            res["span"] = int(cols[-1] - cols[0]) + 1 if cols.numel() else 0
            res["after"] = bool(torch.equal(call(), want)) and wq.wq_last_device_error() == 0
            out.append(res)
        assert short.wq_test_give_up_i8(-1, 0, 0, 0) == 0
        q.put(out)
    except Exception as e:  # noqa: BLE001
        q.put(repr(e))


def _run(cases):
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    pr = ctx.Process(target=_child, args=(q, cases))
    pr.start()
    res = q.get(timeout=300)
    pr.join(60)
    assert isinstance(res, list), res
    assert len(res) == len(cases)
    for r in res:
        assert r["call"] == 0 and r["error"] == 8 and r["then"] == 0, r
        assert r["wrong"] == 0 and r["after"], r
    return res


@pytest.mark.parametrize("name", SPLIT)
def test_split_kernel_gives_up(name):
    """One tile of weight rows is left out, for all tokens, and nothing else."""
    gated, M, N, K = SPLIT[name]
    waits = SPLIT_WAITS + (CLUSTER_WAITS if name.startswith("clusters") else [])
    for r in _run([((gated, M, N, K), w) for w in waits]):
        assert r["rows"] == M and 0 < r["cols"] == r["span"] <= 128 and r["missing"] == M * r["cols"], r
        assert r["first col"] == 2 * r["cols"], r


# three tiles a pair; one
PAIR = {"three tiles": (False, 520, 18944, 2048), "three tiles gated": (True, 520, 9472, 2048),
        "one tile": (False, 300, 4096, 4096), "one tile gated": (True, 300, 4096, 4096)}
# Either CTA's copies stop first, so that the other has some in flight that its peer has not come to; the MMAs stop
# at the first stage, inside a tile, at a tile's start; an epilogue leaves its first and its last accumulator
PAIR_WAITS = [(EMPTY, 5, 0, 20), (EMPTY, 5, 1, 20), (EMPTY, 5, 0, 10), (EMPTY, 5, 1, 10), (FULL, 5, 0, 0),
              (FULL, 5, 0, 13), (DONE, 5, 0, 0), (DONE, 5, 1, 0)]
TILES_WAITS = [(FULL, 5, 0, 32), (FULL, 5, 0, 47), (ACC_EMPTY, 5, 0, 2), (DONE, 5, 0, 1), (DONE, 5, 1, 2),
               (EMPTY, 5, 0, 47), (EMPTY, 5, 1, 47)]


@pytest.mark.parametrize("name", PAIR)
def test_pair_kernel_gives_up(name):
    """Tiles of the one pair are left out, and nothing else; both CTAs' copies have landed when it ends.
    (Of 300 tokens pair 5 has those from 256 on, and its second CTA, whose rows start at 384, none to leave out.)"""
    gated, M, N, K = PAIR[name]
    waits = PAIR_WAITS + (TILES_WAITS if name.startswith("three") else [])
    for w, r in zip(waits, _run([((gated, M, N, K), w) for w in waits])):
        assert r["cols"] <= 3 * 256, (w, r)
        assert (r["missing"] > 0) == (M > 384 or w != (DONE, 5, 1, 0)), (w, r)
