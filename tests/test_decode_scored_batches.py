"""pa_decode_scored where the units (a sequence's K/V heads) outnumber the workers that share them."""

import numpy as np
import pytest

from paged_kv_cache_63_gb300 import lib
from tests.gpu_util import torch
from tests.scored_reference import Cached, Rule, assert_within, attend, slopes_of
from tests.test_decode_scored import P_ERROR, P_FLOOR, gpu_decode

gpu = pytest.mark.gpu

HEADS = {
    "g2": dict(qh=4, kvh=2, hd=64, ps=16),
    "g12": dict(qh=12, kvh=1, hd=64, ps=8),  # two units a K/V head
    "g1": dict(qh=8, kvh=8, hd=128, ps=32),
    "g5": dict(qh=15, kvh=3, hd=128, ps=16),
    "g6": dict(qh=12, kvh=2, hd=256, ps=16),
}


def lengths(n, longest, seed):
    """Many short contexts, empty ones and ones that see nothing among them, and a few long ones."""
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, 40, n)
    ctx[rng.integers(0, n, 4)] = longest
    first = np.where(rng.random(n) < 0.2, ctx + 3, np.minimum(rng.integers(0, 20, n), ctx))
    return ctx, first


@gpu
@pytest.mark.parametrize("workers", [1, 5, 40])
@pytest.mark.parametrize("heads", sorted(HEADS))
def test_few_workers(heads, workers):
    """Units whole in one worker, cut once, and cut over many workers."""
    ctx, first = lengths(70, 900, workers)
    w = Cached(ctx, seed=workers, **HEADS[heads])
    for rule in (Rule(softcap=5.0), Rule(first=first, slopes=slopes_of(w.query_heads)),
                 Rule(window=21)):
        want = attend(w, rule, P_ERROR, P_FLOOR)
        for per_cta in (0, 1, 4):
            opts = lib.options(schedule="balanced", workers=workers, warps_per_cta=per_cta)
            got, flags = gpu_decode(w, rule, opts=opts)
            assert flags == 0
            assert_within(got, *want, False)


@gpu
@pytest.mark.parametrize("heads,n", [("g2", 2100), ("g1", 1030), ("g6", 800)])
def test_many_sequences(heads, n):
    ctx, first = lengths(n, 700, n)
    w = Cached(ctx, seed=n, **HEADS[heads])
    plan = lib.pa_plan(w.prob(), lib.options(schedule="balanced"))
    assert plan["units"] > plan["workers"]
    for rule in (Rule(softcap=5.0), Rule(first=first)):
        got, flags = gpu_decode(w, rule, "fp16", lib.options(schedule="balanced"))
        assert flags == 0
        assert_within(got, *attend(w, rule, P_ERROR, P_FLOOR), True)


@gpu
def test_time_grows_with_the_batch_not_with_its_square():
    """Eight times the sequences take at most twice eight times as long (they took 27 times)."""
    t = torch()
    took = {}
    for n in (512, 4096):
        ps, tokens, maxp = 16, 64, 256
        k, v = (t.randn(n * 4, ps, 8, 128, device="cuda", dtype=t.float16) for _ in range(2))
        q = t.randn(n, 64, 128, device="cuda", dtype=t.float16)
        bt = t.zeros(n, maxp, device="cuda", dtype=t.int32)
        bt[:, :4] = t.randperm(n * 4, device="cuda").view(n, 4)
        ctx = t.full((n,), tokens, device="cuda", dtype=t.int32)
        prob = lib.problem(n, 64, 8, 128, ps, maxp, n * 4)
        size = lib.pa_workspace_size(prob)
        ws = t.empty(size, dtype=t.uint8, device="cuda")
        out = t.empty(n, 64, 128, device="cuda")
        best = float("inf")
        for _ in range(8):
            a, b = (t.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            lib.pa_decode_scored(prob, None, q, k, v, bt, ctx, 0.1, out, workspace=ws,
                                 workspace_bytes=size)
            b.record()
            t.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        assert lib.pa_get_device_error() == 0
        took[n] = best
    assert took[4096] <= 16 * took[512], took
