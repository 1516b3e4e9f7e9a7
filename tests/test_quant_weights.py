"""Weights of tokens whose values have small scales beside seen tokens whose values have large ones:
pa_decode_quant and the few rows of pa_prefill_quant hold every weight to the same bits, whatever the
scales around it."""

import numpy as np
import pytest

from tests.gpu_util import torch
from tests.quant_reference import QuantCached, quantise
from tests.scored_reference import Rule, assert_within, attend, seen, slopes_of
from tests.test_decode_quant import SHAPES, gpu_decode, redo
from tests.test_prefill_quant import few, gpu_prefill

gpu = pytest.mark.gpu

# A weight meets V as fp16 and its remainder in fp16: 2^-22 of it (11 bits each). The remainder is told
# from 0 down to 2^-25, and the largest weight is at least 2^7, so a weight is off by no more than 2^-32
# of the largest, nor by more than itself.
P_ERROR, FLOOR = 2.0 ** -22, 2.0 ** -32


def formula(w, rule):
    """attend's (out, bound) with that floor for each token by itself."""
    out, bound = attend(w, rule, P_ERROR, 0.0)
    g = w.query_heads // w.kv_heads
    for b in range(w.batch):
        keys, values = [x.astype(np.float64) for x in w.gathered(b)]
        for row, pos in w.rows_of(b):
            lo, end = seen(rule, b, row, pos, int(w.ctx[b]))
            for h in range(w.query_heads if lo < end else 0):
                s = w.scale * (keys[lo:end, h // g] @ w.q[row, h].astype(np.float64))
                if rule.softcap:
                    s = rule.softcap * np.tanh(s / rule.softcap)
                if rule.slopes is not None:
                    s = s - float(rule.slopes[h]) * np.abs(pos - np.arange(lo, end))
                p = np.exp(s - s.max())
                off = np.minimum(p, FLOOR) / p.sum()
                bound[row, h] += off @ np.abs(values[lo:end, h // g]) + off.sum() * np.abs(out[row, h])
    return out, bound


def put(w, name, b, t, x, exponent=None):
    """Token t's row [kv_head][head_dim]; with an exponent, its codes under that power of two."""
    at = w.bt[b, t // w.ps], t % w.ps
    codes, scales = quantise(x)
    if exponent is not None:
        scales = np.full_like(scales, 127 + exponent)
    getattr(w, name + "_codes")[at], getattr(w, name + "_scales")[at] = codes, scales


def make(shape, ctx, heavy, apart, new=None):
    """Tokens `heavy` (distances from the end) of each sequence carry all the weight, in shares that
    are no powers of two, under values of scale 2^-15; the others' values have 2^(apart - 15), and
    their weight is less than 2^-100."""
    w = QuantCached(ctx, new, seed=11, **SHAPES[shape])
    rng = np.random.default_rng(12)
    kvh, hd = w.kv_heads, w.head_dim
    u = rng.choice([-1.0, 1.0], (kvh, hd))
    for b, n in enumerate(w.ctx):
        for t in range(int(n)):
            place = heavy.index(n - 1 - t) if n - 1 - t in heavy else None
            score = -(8.0 + rng.integers(0, 4)) if place is None else -0.007 * place
            put(w, "k", b, t, u * score)
            row = rng.uniform(100, 240, (kvh, hd))
            row[:, 0] = 240  # (so that no code is above 240, the most that 2^8 takes)
            row *= rng.choice([-1, 1], (kvh, hd))
            put(w, "v", b, t, row, -15 + (apart if place is None else 0))
    size = rng.uniform(1.0, 1.5, (w.rows, w.query_heads, 1))
    w.q = (size * np.repeat(u, w.query_heads // kvh, axis=0)).astype(np.float16)
    w.scale = 1.0 if hd == 64 else 0.5 if hd == 128 else 0.25
    redo(w)
    return w


@gpu
@pytest.mark.parametrize("apart", [3, 12, 16, 20, 23])
@pytest.mark.parametrize("shape", ["hd64_g2", "hd64_g1", "hd128_g4", "hd128_g16", "hd256_g6", "hd256_g1"])
def test_decode_weights_beside_large_scales(shape, apart):
    for ctx, heavy in (([40, 7, 200], [3, 5]), ([129, 65], [0, 17, 33, 34, 35]), ([33, 600], [6])):
        w = make(shape, ctx, heavy, apart)
        for rule in (Rule(), Rule(softcap=50.0, slopes=0.001 * slopes_of(w.query_heads))):
            got, flags = gpu_decode(w, rule)
            assert flags == 0
            assert_within(got, *formula(w, rule), False)


@gpu
@pytest.mark.parametrize("apart", [3, 16, 23])
@pytest.mark.parametrize("shape", ["hd64_g1", "hd128_g4", "hd256_g6"])
def test_few_rows_weights_beside_large_scales(shape, apart):
    """The newest tokens' values are large: they share tiles, and eight rows' walk, with rows that do
    not see them."""
    for ctx, new, heavy in (([40, 200], [2, 1], [3, 5]), ([130, 65], [3, 3], [4, 17, 33])):
        w = make(shape, ctx, heavy, apart, new)
        assert few(w, Rule(), max(new))
        got, flags = gpu_prefill(w, Rule())
        assert flags == 0
        assert_within(got, *formula(w, Rule()), True)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_values_of_the_whole_range_of_scales(shape):
    """Exponents of -15 .. 8 over every tile, weights of all sizes."""
    w = QuantCached([200, 47, 130], seed=6, q_scale=2.0, **SHAPES[shape])
    rng = np.random.default_rng(3)
    live = np.isfinite(w.v[..., 0])
    w.v_scales[live] = 127 + rng.integers(-15, 8, int(live.sum()))
    redo(w)
    for rule in (Rule(), Rule(window=60)):
        got, flags = gpu_decode(w, rule)
        assert flags == 0
        assert_within(got, *formula(w, rule), False)


def test_inputs_are_what_they_say():
    w = make("hd128_g4", [40, 200], [3, 5], 23)
    assert torch() is not None
    for b, n in enumerate(w.ctx):
        keys, values = [x.astype(np.float64) for x in w.gathered(b)]
        s = w.scale * (keys[:, 0] @ w.q[b, 0].astype(np.float64))
        order = np.argsort(-s)
        assert sorted(order[:2].tolist()) == [n - 6, n - 4] and s[order[2]] < s[order[1]] - 80
        share = np.exp(s[order[1]] - s[order[0]])
        assert 0.5 < share < 0.999
        assert np.abs(values[order[:2]]).max() < 2.0 ** -6 and np.abs(values[order[2:]]).min() > 1000
