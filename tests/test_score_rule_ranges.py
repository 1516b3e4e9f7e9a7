"""The score rule over the ranges of its fields and the caches: caps far above and far below every
score, rows of very different scores side by side, cached values next to fp16's largest."""

import numpy as np
import pytest

from paged_kv_cache_63_gb300 import lib
from tests.scored_reference import Cached, Rule, assert_within, attend, slopes_of
from tests.test_decode_scored import P_ERROR, P_FLOOR, gpu_decode
from tests.test_prefill_scored import ERRORS, SHAPES, documents, gpu_prefill

gpu = pytest.mark.gpu

KERNELS = ["hd64_g2", "hd128_g4", "hd256_g6"]


def chunks(shape, **kw):
    args = dict(ctx=[300, 1, 129, 200], new=[170, 1, 60, 31], q_scale=3.0, seed=11, pad=3)
    args.update(SHAPES[shape])
    args.update(kw)
    return Cached(args.pop("ctx"), args.pop("new"), **args)


def check_prefill(w, rule, **errors):
    got, flags = gpu_prefill(w, rule)
    assert flags == 0
    want, bound = attend(w, rule, **dict(ERRORS, **errors))
    assert np.isnan(got[np.isnan(want)]).all()
    assert_within(got, want, bound, True)


@gpu
@pytest.mark.parametrize("softcap", [1e4, 1e5, 1e6, 1e9, 1e30])
@pytest.mark.parametrize("shape", KERNELS)
def test_caps_far_above_the_scores(shape, softcap):
    """Such a cap changes next to nothing. The bound of the other multi-token tests holds: tanh's
    argument, its square, three steps of the polynomial, the cap and their products are off by
    2^-24 each, seven in all (4.2e-7 beside the polynomial's 5.8e-7, of the 1.1e-6 that
    `cap_error` and the scaled score's 2^-22 allow)."""
    w = chunks(shape)
    slopes = slopes_of(w.query_heads)
    for rule in (Rule(softcap=softcap), Rule(softcap=softcap, window=70),
                 Rule(softcap=softcap, slopes=slopes),
                 Rule(softcap=softcap, first=documents(w, 40)),
                 Rule(softcap=softcap, slopes=slopes, first=documents(w, 90),
                      prefix=np.array([200, 0, 80, 0]))):
        check_prefill(w, rule)
    step = Cached([300, 1, 129, 17], q_scale=3.0, seed=11, **SHAPES[shape])
    got, flags = gpu_decode(step, Rule(softcap=softcap))
    assert flags == 0
    assert_within(got, *attend(step, Rule(softcap=softcap), P_ERROR, P_FLOOR), False)


@gpu
@pytest.mark.parametrize("softcap", [1e-3, 1e-12, 1e-30])
@pytest.mark.parametrize("shape", KERNELS)
def test_caps_far_below_the_scores(shape, softcap):
    """Every score is next to the cap, and all seen tokens weigh nearly the same."""
    w = chunks(shape)
    check_prefill(w, Rule(softcap=softcap))
    check_prefill(w, Rule(softcap=softcap, window=70, slopes=slopes_of(w.query_heads)))


def test_caps_without_a_normal_quotient_are_refused():
    prob = lib.problem(4, 32, 8, 128, 16, 256, 1024)
    at = 1 << 20
    for softcap in (1e-45, 1e-39, 5e-40, 3e38):  # the scale is 0.1
        s = lib.score(softcap=softcap, out="fp16")
        assert lib.status_of(lib.pa_prefill_scored, prob, s, at, at, 100, 50, at, at, at, at, 0.1,
                             at) == 1
        assert lib.status_of(lib.pa_decode_scored, prob, s, at, at, at, at, at, 0.1, at) == 1


@gpu
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("softcap", [20.0, 256.0, 300.0, 5e4])
@pytest.mark.parametrize("shape", KERNELS)
def test_small_scores_beside_large_ones(shape, softcap, biased):
    """Rows whose scores pass the cap's half leave the small scores of the rows beside them as exact
    as they are alone; up to a cap of 256 as exact as 1 - 2 / (1 + e^2t) is: half of 2^-22 and of
    the 2^-23 of the exponential's argument, 2^-23 + 2^-24 of the reciprocal and its sum, 2^-24 of
    the result, 3.6e-7 of the cap in all."""
    w = chunks(shape)
    signs = np.sign(w.q[::16].astype(np.float32))
    w.q[::16] = (signs * 0.5 * softcap).astype(np.float16)
    off = 3.6e-7 * softcap if softcap <= 256 else 0.0
    check_prefill(w, Rule(softcap=softcap, slopes=slopes_of(w.query_heads) if biased else None),
                  probability_error=ERRORS["probability_error"] + off)


@gpu
@pytest.mark.parametrize("shape", KERNELS)
def test_values_next_to_the_largest_of_fp16(shape):
    """A mean of finite values is finite: the weights' rounding must not carry it past them."""
    for w in (chunks(shape, ctx=[64, 40, 3], new=[64, 9, 3]),
              chunks(shape, ctx=[300], new=[300], q_scale=0.3)):
        sign = np.where(np.arange(w.head_dim) % 2, -1.0, 1.0)
        w.v[np.isfinite(w.v)] = 1.0
        w.v = (w.v * (65504.0 * sign)).astype(np.float16)
        for rule in (Rule(), Rule(softcap=20.0), Rule(window=3),
                     Rule(slopes=slopes_of(w.query_heads))):
            check_prefill(w, rule)
    step = Cached([64, 40, 3, 300], q_scale=3.0, seed=12, **SHAPES[shape])
    step.v[np.isfinite(step.v)] = 65504.0
    got, flags = gpu_decode(step, Rule(softcap=20.0), "fp16")
    assert flags == 0
    assert_within(got, *attend(step, Rule(softcap=20.0), P_ERROR, P_FLOOR), True)
