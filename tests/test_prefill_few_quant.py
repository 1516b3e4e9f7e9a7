"""pa_prefill_quant where there are few rows (new tokens by query heads of a K/V head): the kernel that
shares a row's keys between warps, against the formula in 64 bits. Probabilities are as the decode
step's, so its bounds hold."""

import numpy as np
import pytest

from paged_kv_cache_63_gb300 import lib
from tests.gpu_util import torch
from tests.quant_reference import QuantCached
from tests.scored_reference import Rule, assert_within, attend, device_rule, slopes_of
from tests.test_decode_quant import formula
from tests.test_prefill_quant import few, gpu_prefill

gpu = pytest.mark.gpu

SHAPES = {
    "hd64_g2": dict(qh=4, kvh=2, hd=64, ps=16),
    "hd64_g1": dict(qh=3, kvh=3, hd=64, ps=8),
    "hd128_g4": dict(qh=8, kvh=2, hd=128, ps=16),
    "hd128_g3": dict(qh=6, kvh=2, hd=128, ps=8),
    "hd128_g32": dict(qh=32, kvh=1, hd=128, ps=256),
    "hd256_g6": dict(qh=12, kvh=2, hd=256, ps=64),
    "hd256_g1": dict(qh=1, kvh=1, hd=256, ps=16),
}


def case(shape, ctx=(300, 5, 129, 0, 1, 1000, 40), seed=1, **kw):
    s = SHAPES[shape]
    most = 32 // (s["qh"] // s["kvh"])
    ctx = np.asarray(ctx)
    new = np.minimum(ctx, np.array([most, max(1, most // 2), 1, 0, 1, most, 0])[:len(ctx)])
    return QuantCached(ctx, new, q_scale=3.0, seed=seed, pad=3, **{**s, **kw})


def check(w, rule, **kw):
    assert few(w, rule, kw.get("max_query_len") or int(w.new.max()))
    got, flags = gpu_prefill(w, rule, **kw)
    assert flags == 0
    want, bound = formula(w, rule)
    assert np.isnan(got[np.isnan(want)]).all()  # rows of no new token are left alone
    return assert_within(got, want, bound, True)


def rules(w):
    qh = w.query_heads
    return {
        "none": Rule(),
        "cap": Rule(softcap=2.0),
        "cap_wide": Rule(softcap=400.0),
        "window1": Rule(window=1),
        "window5": Rule(window=5),
        "window130": Rule(window=130),
        "slopes": Rule(slopes=slopes_of(qh)),
        "prefix": Rule(prefix=np.array([290, 5, 129, 0, 1, 1 << 30, -4])),
        "prefix_slopes": Rule(prefix=np.array([300, 2, 0, 9, 0, 990, 40]), slopes=slopes_of(qh)),
        "all": Rule(softcap=3.0, window=90, slopes=slopes_of(qh),
                    prefix=np.array([299, 4, 129, 0, 1, 995, 3])),
    }


@gpu
@pytest.mark.parametrize("rule", sorted(rules(case("hd64_g2"))))
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_matches_formula(shape, rule):
    w = case(shape, head_major=len(shape + rule) % 2)
    check(w, rules(w)[rule])


@gpu
@pytest.mark.parametrize("shape", ["hd64_g1", "hd128_g3", "hd256_g1"])
def test_more_tokens_of_one_sequence(shape):
    """A short prompt, and a chunk on a prefix: many CTAs of one sequence, the last with few rows."""
    for ctx, new in ([133, 133], [500, 61], [9, 9]):
        w = QuantCached([ctx], [new], q_scale=3.0, seed=2, **SHAPES[shape])
        check(w, Rule())
        check(w, Rule(window=40, softcap=9.0, prefix=np.array([ctx - 3])))
        check(w, Rule(slopes=slopes_of(w.query_heads)), max_query_len=new + 5)


@gpu
@pytest.mark.parametrize("new", [1, 9, 30, 70, 150])
@pytest.mark.parametrize("shape", ["hd64_g1", "hd128_g3", "hd128_g32", "hd256_g6", "hd256_g1"])
def test_keys_shared_by_a_cluster(shape, new):
    """One long context, so that the blocks of a cluster (two to eight of them, fewer with more rows)
    share its keys; alone, and beside a short one, for which most of them have none."""
    for ctx in ([2500], [2300, 5]):
        n = [min(new, x) for x in ctx]
        w = QuantCached(ctx, n, q_scale=3.0, seed=2, head_major=new % 2, pad=2, **SHAPES[shape])
        if not few(w, Rule(), max(n)):
            continue
        check(w, Rule())
        check(w, Rule(window=700, softcap=9.0, slopes=slopes_of(w.query_heads)))
        for b in range(w.batch):
            w.forget(b, max(0, int(w.ctx[b] - w.new[b]) - 64 + 1))
        got, flags = gpu_prefill(w, Rule(window=64))
        assert flags == 0
        # (the formula does not read what the window hides)
        assert_within(got, *formula(w, Rule(window=64)), True)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g1", "hd128_g3", "hd256_g1"])
def test_clusters_replayed_expired_and_at_once(shape):
    t = torch()
    w = QuantCached([3000], [4], seed=6, **SHAPES[shape])
    want = formula(w, Rule())
    d, dr = w.to_device(), device_rule(Rule(), "fp16")
    outs = [t.zeros(w.rows, w.query_heads, w.head_dim, device="cuda", dtype=t.float16)
            for _ in range(3)]
    streams = [t.cuda.Stream() for _ in outs]
    t.cuda.synchronize()
    for _ in range(5):
        for o, s in zip(outs, streams):
            lib.pa_prefill_quant(w.prob(), dr, d["q"], d["qs"], w.rows, 4, d["cache"], d["bt"], d["ctx"],
                                 w.scale, o, stream=s)
    t.cuda.synchronize()
    first = outs[0].cpu().numpy()
    assert_within(first, *want, True)
    assert all(np.array_equal(o.cpu().numpy(), first) for o in outs)
    _, flags = gpu_prefill(w, Rule(), lib.options(test_flags=lib.PA_TEST_EXPIRE_WAITS))
    assert flags == lib.PA_DEVERR_TIMEOUT
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        lib.pa_prefill_quant(w.prob(), dr, d["q"], d["qs"], w.rows, 4, d["cache"], d["bt"], d["ctx"],
                             w.scale, outs[1])
    for _ in range(3):
        outs[1].zero_()
        g.replay()
        t.cuda.synchronize()
        assert np.array_equal(outs[1].cpu().numpy(), first)
    assert lib.pa_get_device_error() == 0


@gpu
@pytest.mark.parametrize("shape", ["hd64_g1", "hd128_g4"])
def test_many_sequences_of_few_rows(shape):
    rng = np.random.default_rng(6)
    ctx = rng.integers(0, 70, 400)
    w = QuantCached(ctx, np.minimum(ctx, rng.integers(0, 3, 400)), seed=3, **SHAPES[shape])
    check(w, Rule(window=30))


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_single_tokens_agree_with_the_decode_step(shape):
    from tests.test_decode_quant import gpu_decode

    ctx = [300, 1, 129, 16, 700]
    w = QuantCached(ctx, [1] * 5, **SHAPES[shape])
    got, flags = gpu_prefill(w, Rule(softcap=5.0))
    assert flags == 0
    one = QuantCached(ctx, **SHAPES[shape])
    assert np.array_equal(one.q, w.q) and np.array_equal(one.k_codes, w.k_codes)
    step, _ = gpu_decode(one, Rule(softcap=5.0), "fp16")
    want, bound = formula(one, Rule(softcap=5.0))
    assert_within(got, want, bound, True)
    assert (np.abs(got.astype(np.float64) - step)
            <= 2 * bound + (np.abs(want) + bound) * 2.0 ** -10 + 2.0 ** -24).all()


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
@pytest.mark.parametrize("window", [1, 33, 200])
def test_tokens_nobody_sees_are_never_read(shape, window):
    w = case(shape)
    rule = Rule(window=window, softcap=10.0)
    want = formula(w, rule)
    for b in range(w.batch):
        w.forget(b, max(0, int(w.ctx[b] - w.new[b]) - window + 1))
    got, flags = gpu_prefill(w, rule)
    assert flags == 0
    assert_within(got, *want, True)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_bits_do_not_depend_on_what_is_not_seen(shape):
    w = case(shape)
    rows, outs = int(w.qs[-1]), []
    for fill, code, scale in ((0.0, 0, 127), (3000.0, 0x7e, 135), (np.nan, 0x7f, 255)):
        for x in "kv":
            unseen = ~np.isfinite(getattr(w, x)[..., 0])
            getattr(w, x + "_codes")[unseen] = code
            getattr(w, x + "_scales")[unseen] = scale
        w.q[rows:] = fill
        out, flags = gpu_prefill(w, Rule(softcap=20.0, slopes=slopes_of(w.query_heads)))
        assert flags == 0
        outs.append(out[:rows].view(np.uint16))
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_scales_of_the_whole_range_and_growing_maxima(shape):
    from tests.test_decode_quant import redo

    w = case(shape)
    for b in range(w.batch):
        n = int(w.ctx[b])
        for t in range(n):
            at = w.bt[b, t // w.ps], t % w.ps
            w.k_scales[at] = 127 - 12 + 5 * t // n
            w.v_scales[at] = 127 - 15 + 23 * ((t * 7) % n) // n
    w.spread = 23
    redo(w)
    check(w, Rule())
    check(w, Rule(window=150))
    w.scale = -w.scale
    check(w, Rule(softcap=20.0))
    w.scale = 0.0
    check(w, Rule())
    check(w, Rule(softcap=20.0))


@gpu
def test_replayed_at_once_and_deterministic():
    t = torch()
    w = case("hd128_g4", ctx=(3000, 5, 129, 0, 1, 2000, 40))
    rule = Rule(softcap=8.0, window=2500)
    want = formula(w, rule)
    d, dr = w.to_device(), device_rule(rule, "fp16")
    outs = [t.zeros(w.rows, 8, 128, device="cuda", dtype=t.float16) for _ in range(2)]
    call = lambda o: lib.pa_prefill_quant(  # noqa: E731
        w.prob(), dr, d["q"], d["qs"], w.rows, 8, d["cache"], d["bt"], d["ctx"], w.scale, o)
    graphs = []
    for o in outs:
        call(o)
        t.cuda.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            call(o)
        graphs.append((g, t.cuda.Stream()))
    live = ~np.isnan(want[0])
    first = outs[0].cpu().numpy()
    assert_within(first, *want, True)
    for _ in range(5):
        for o in outs:
            o.fill_(0)
        t.cuda.synchronize()
        for g, s in graphs:
            with t.cuda.stream(s):
                g.replay()
        t.cuda.synchronize()
        for o in outs:
            got = o.cpu().numpy()
            assert np.array_equal(got[live], first[live]) and (got[~live] == 0).all()
    assert lib.pa_get_device_error() == 0


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd256_g6"])
def test_bad_inputs_are_flagged_and_expired_waits_reported(shape):
    t = torch()
    w = case(shape)
    d, rule = w.to_device(), Rule(window=150)
    want = formula(w, rule)
    qs, ctx = w.qs.tolist(), w.ctx.tolist()
    for name, value, flag in [
            ("ctx", [-1] + ctx[1:], lib.PA_DEVERR_CONTEXT),
            ("ctx", [w.maxp * w.ps + 1] + ctx[1:], lib.PA_DEVERR_CONTEXT),
            ("ctx", [1] + ctx[1:], lib.PA_DEVERR_QUERY_START),
            ("qs", qs[:-1] + [9999], lib.PA_DEVERR_QUERY_START)]:
        bad = dict(d, **{name: t.tensor(value, dtype=t.int32, device="cuda")})
        got, flags = gpu_prefill(w, rule, d=bad)
        assert flags == flag
        other = slice(qs[1], qs[6])
        assert_within(got[other], want[0][other], want[1][other], True)
        if name == "ctx":
            assert np.isnan(got[:qs[1]]).all()
    _, flags = gpu_prefill(w, rule, lib.options(test_flags=lib.PA_TEST_EXPIRE_WAITS))
    assert flags == lib.PA_DEVERR_TIMEOUT
    check(w, rule)
    w.bt[0, -1 if w.maxp * w.ps == 300 else 299 // w.ps] = w.pages
    got, flags = gpu_prefill(w, rule)
    assert flags == lib.PA_DEVERR_PAGE_ID
    other = slice(qs[1], qs[6])
    assert_within(got[other], want[0][other], want[1][other], True)
