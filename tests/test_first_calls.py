"""A process's first calls, made by several threads at once under different plans."""

import subprocess
import sys

import pytest

from tests.conftest import ROOT

PROGRAM = r"""
import sys, threading
import numpy as np
import torch as t
from paged_kv_cache_63_gb300 import lib
from tests.gpu_util import assert_close
from tests.scored_reference import Cached, Rule, assert_within, attend, device_rule

hd, scored = int(sys.argv[1]), sys.argv[2] == "scored"
w = Cached([900, 33, 400], qh=8, kvh=2, hd=hd, ps=16, seed=1)
rule = Rule(softcap=5.0) if scored else Rule()
want = attend(w, rule, 2.0 ** -22, 2.0 ** -32)
d, dr, prob = w.to_device(), device_rule(rule, "fp32"), w.prob()
plans = [dict(stages=s, warps_per_cta=n) for s in (1, 2) for n in (1, 2, 4, 6)]
work = []
for plan in plans:
    opts = lib.options(schedule="balanced", **plan)
    n = lib.pa_workspace_size(prob, opts)
    assert n > 0
    work.append((opts, t.zeros(n, dtype=t.uint8, device="cuda"), n, t.cuda.Stream(),
                 t.full((3, 8, hd), float("nan"), device="cuda")))
t.cuda.synchronize()
start, failed = threading.Barrier(len(work)), []


def call(opts, ws, n, stream, out):
    start.wait()
    try:
        for _ in range(3):
            if scored:
                lib.pa_decode_scored(prob, dr, d["q"], d["k"], d["v"], d["bt"], d["ctx"], w.scale,
                                     out, opts, ws, n, stream=stream.cuda_stream)
            else:
                lib.pa_decode_ex(prob, d["q"], d["k"], d["v"], d["bt"], d["ctx"], w.scale, out,
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
for *_, out in work:
    if scored:
        assert_within(out.cpu().numpy(), *want, False)
    else:
        assert_close(out.cpu().numpy(), want[0])
print("ok")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["scored", "plain"])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_first_calls_at_once(hd, call):
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(hd), call], cwd=ROOT, timeout=300,
                       capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
