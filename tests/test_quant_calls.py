"""The calls on a quantised cache as programs make them: from threads, as a process's first, in large
batches, over shared pages; and the binding's checks of their tensors."""

import subprocess
import sys
import threading

import numpy as np
import pytest

from paged_kv_cache_63_gb300 import lib
from tests.conftest import ROOT
from tests.gpu_util import torch
from tests.quant_reference import QuantCached
from tests.scored_reference import Rule, assert_within, attend
from tests.test_append_rope import table_of

gpu = pytest.mark.gpu


def entry_points(w):
    """Name: (call, its outputs) over the inputs of w, one new token to a sequence."""
    t = torch()
    d, prob = w.to_device(), w.prob()
    b, qh, kvh, hd = w.batch, w.query_heads, w.kv_heads, w.head_dim
    half = lambda *s: t.zeros(*s, hd, dtype=t.float16, device="cuda")  # noqa: E731
    n = lib.pa_quant_workspace_size(prob)
    ws = t.empty(n, dtype=t.uint8, device="cuda")
    qs = t.arange(b + 1, dtype=t.int32, device="cuda")
    kv = [t.randn(b, kvh, hd, device="cuda").half() for _ in range(2)]
    written = [d[x].clone() for x in ("kc", "vc", "ks", "vs")]
    rope = lib.rope(hd, "half", t.from_numpy(table_of(int(w.ctx.max()), hd)).cuda())
    norm = lib.norm(1e-6, t.ones(hd, device="cuda"), t.ones(hd, device="cuda"))
    score = lib.score(softcap=5.0, out="fp16")
    q_out, dec, pre, many = (half(b, qh) for _ in range(4))
    k, v = half(b, kvh), half(b, kvh)
    return {
        "append": (lambda: lib.pa_append_quant(prob, norm, rope, d["q"], *kv, qs, b, d["bt"], d["ctx"],
                                               q_out, lib.quant_cache(*written)), [q_out, *written]),
        "read": (lambda: lib.pa_read_quant(prob, d["cache"], qs, b, d["bt"], d["ctx"], k, v), [k, v]),
        "decode": (lambda: lib.pa_decode_quant(prob, score, d["q"], d["cache"], d["bt"], d["ctx"],
                                               w.scale, dec, workspace=ws, workspace_bytes=n), [dec]),
        "prefill": (lambda: lib.pa_prefill_quant(prob, score, d["q"], qs, b, 1, d["cache"], d["bt"],
                                                 d["ctx"], w.scale, pre), [pre]),
        # (a grid for many rows)
        "prefill_many": (lambda: lib.pa_prefill_quant(prob, score, d["q"], qs, b, 2500, d["cache"],
                                                      d["bt"], d["ctx"], w.scale, many), [many]),
    }


@gpu
@pytest.mark.parametrize("head_major", [0, 1])
def test_a_threads_first_call(head_major):
    t = torch()
    for name, (call, outs) in entry_points(QuantCached([700, 33], head_major=head_major)).items():
        call()
        t.cuda.synchronize()
        want = [x.clone() for x in outs]
        for x in outs:
            x.zero_()
        t.cuda.synchronize()
        failed = []

        def first():
            try:
                call()
            except lib.PagedAttnError as e:
                failed.append(e)

        thread = threading.Thread(target=first)
        thread.start()
        thread.join()
        t.cuda.synchronize()
        assert not failed, (name, failed)
        if name != "append":  # (its other slots were zeroed with the rows)
            assert all(t.equal(a.view(t.uint8), b.view(t.uint8)) for a, b in zip(outs, want)), name
        else:
            assert t.equal(outs[0], want[0])
            assert all(bool((b[a != 0] == a[a != 0]).all()) and bool((a != 0).any())
                       for a, b in zip(outs[1:], want[1:]))
        assert lib.pa_get_device_error() == 0


PROGRAM = r"""
import sys, threading
import numpy as np
import torch as t
from paged_kv_cache_63_gb300 import lib
from tests.quant_reference import QuantCached
from tests.scored_reference import Rule, assert_within, attend, device_rule

hd = int(sys.argv[1])
w = QuantCached([900, 33, 400], qh=8, kvh=2, hd=hd, ps=16, seed=1)
rule = Rule(softcap=5.0)
want = attend(w, rule, 2.0 ** -22, 2.0 ** (w.spread + 2 - 32))
d, dr, prob = w.to_device(), device_rule(rule, "fp32"), w.prob()
half = device_rule(rule, "fp16")
qs = t.arange(4, dtype=t.int32, device="cuda")
work = []
for plan in [dict(stages=s, warps_per_cta=n) for s in (1, 2) for n in (0, 1, 4)] + [None] * 4:
    opts = None if plan is None else lib.options(schedule="balanced", **plan)
    n = lib.pa_quant_workspace_size(prob, opts)
    out = t.full((3, 8, hd), float("nan"), device="cuda")
    work.append((opts, t.zeros(n, dtype=t.uint8, device="cuda"), n, t.cuda.Stream(),
                 out.half() if opts is None else out))
t.cuda.synchronize()
start, failed = threading.Barrier(len(work)), []


def call(opts, ws, n, stream, out):
    start.wait()
    try:
        for _ in range(3):
            if opts is None:
                # the kernel for few rows, and those for many
                for most in (1, 2500):
                    lib.pa_prefill_quant(prob, half, d["q"], qs, 3, most, d["cache"], d["bt"],
                                         d["ctx"], w.scale, out, stream=stream.cuda_stream)
            else:
                lib.pa_decode_quant(prob, dr, d["q"], d["cache"], d["bt"], d["ctx"], w.scale, out,
                                    opts, ws, n, stream=stream.cuda_stream)
    except Exception as e:
        failed.append(repr(e))


threads = [threading.Thread(target=call, args=a) for a in work]
for x in threads:
    x.start()
for x in threads:
    x.join()
t.cuda.synchronize()
assert not failed, failed
assert lib.pa_get_device_error() == 0
slack = attend(w, rule, 2.0 ** -11, 2.0 ** -25, cap_error=6.3e-7 + 2.0 ** -22, span=128)
for opts, *_, out in work:
    assert_within(out.float().cpu().numpy(), *(slack if opts is None else want), opts is None)
print("ok")
"""


@gpu
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_first_calls_at_once(hd):
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(hd)], cwd=ROOT, timeout=300,
                       capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


@gpu
@pytest.mark.parametrize("shape", [dict(qh=8, kvh=8, hd=64, ps=16), dict(qh=16, kvh=4, hd=128, ps=32),
                                   dict(qh=4, kvh=4, hd=256, ps=16)])
def test_more_units_than_workers(shape):
    """Batches of short contexts, some empty, alone and with long ones among them."""
    from tests.test_decode_quant import check

    rng = np.random.default_rng(4)
    for ctx in (rng.integers(0, 90, 700), np.where(rng.random(500) < 0.01, 700,
                                                   rng.integers(0, 40, 500))):
        w = QuantCached(ctx, seed=3, **shape)
        check(w, Rule(window=50, softcap=9.0))
        check(w, Rule(), "fp16")


@gpu
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_sequences_share_pages(hd):
    """A prefix that several sequences' tables name, and a page that one table names twice."""
    from tests.test_decode_quant import formula, gpu_decode
    from tests.test_prefill_quant import ERRORS, gpu_prefill

    w = QuantCached([100, 100, 100, 64], hd=hd, ps=16, seed=5)
    w.bt[1, :4] = w.bt[2, :4] = w.bt[0, :4]
    w.bt[3, 2] = w.bt[3, 0]
    got, flags = gpu_decode(w, Rule())
    assert flags == 0
    assert_within(got, *formula(w, Rule()), False)
    p = QuantCached([100, 100, 100, 64], [7, 1, 30, 64], hd=hd, ps=16, seed=5)
    p.bt = w.bt
    for x in ("k", "v", "k_codes", "v_codes", "k_scales", "v_scales"):
        setattr(p, x, getattr(w, x))
    got, flags = gpu_prefill(p, Rule())
    assert flags == 0
    assert_within(got, *attend(p, Rule(), **ERRORS), True)


@gpu
def test_binding_refuses_tensors_that_are_too_short_or_of_another_type():
    t = torch()
    w = QuantCached([40, 20])
    d, prob = w.to_device(), w.prob()
    b, qh, kvh, hd = w.batch, w.query_heads, w.kv_heads, w.head_dim
    z = lambda *s, dt=t.float16: t.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    qs = t.arange(b + 1, dtype=t.int32, device="cuda")
    n = lib.pa_quant_workspace_size(prob)
    score, ws = lib.score(out="fp16"), z(n + 256, dt=t.uint8)
    calls = {
        "append": (lambda a: lib.pa_append_quant(prob, None, None, *a[:4], b, *a[4:]),
                   [z(b, qh, hd), z(b, kvh, hd), z(b, kvh, hd), qs, d["bt"], d["ctx"], z(b, qh, hd),
                    d["cache"]]),
        "read": (lambda a: lib.pa_read_quant(prob, a[0], a[1], b, *a[2:]),
                 [d["cache"], qs, d["bt"], d["ctx"], z(b, kvh, hd), z(b, kvh, hd)]),
        "decode": (lambda a: lib.pa_decode_quant(prob, score, *a[:4], w.scale, a[4], workspace=ws,
                                                 workspace_bytes=n),
                   [d["q"], d["cache"], d["bt"], d["ctx"], z(b, qh, hd)]),
        "prefill": (lambda a: lib.pa_prefill_quant(prob, score, a[0], a[1], b, 1, *a[2:5], w.scale,
                                                   a[5]),
                    [d["q"], qs, d["cache"], d["bt"], d["ctx"], z(b, qh, hd)]),
    }
    parts = [d["kc"], d["vc"], d["ks"], d["vs"]]
    for name, (call, args) in calls.items():
        assert lib.status_of(call, args) == 0, name
        for i, x in enumerate(args):
            if x is d["cache"]:
                for j in range(4):
                    short = list(parts)
                    short[j] = parts[j].flatten()[:-1]
                    a = list(args)
                    a[i] = lib.quant_cache(*short)
                    assert lib.status_of(call, a) == 1, (name, "cache", j)
                continue
            for bad in (x.flatten()[:-1], x.to(t.float64)):
                a = list(args)
                a[i] = bad
                with pytest.raises((lib.PagedAttnError, ValueError)):
                    call(a)
    t.cuda.synchronize()
    assert lib.pa_get_device_error() == 0
    with pytest.raises(lib.PagedAttnError):
        lib.quant_cache(d["kc"].transpose(1, 2), *parts[1:])  # not whole
    norm = lib.norm(1e-6, z(hd - 4, dt=t.float32))
    call, args = calls["append"]
    assert lib.status_of(lambda a: lib.pa_append_quant(prob, norm, None, *a[:4], b, *a[4:]), args) == 1
