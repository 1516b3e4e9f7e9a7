"""pa_decode_quant (a decode step over a quantised cache) against the formula in 64 bits over what the
codes stand for, where it can go wrong; refusals on the host."""

import numpy as np
import pytest

from paged_kv_cache_63_gb300 import lib
from tests.gpu_util import torch
from tests.quant_reference import QuantCached
from tests.scored_reference import Rule, assert_within, attend, device_rule, slopes_of
from tests.test_decode_scored import CTX, SHAPES, rules

gpu = pytest.mark.gpu
GOOD = 1 << 20

# A probability times its value's scale meets the codes as fp16 and its remainder in fp16: 22 bits
# of it, the product told from 0 down to 2^-25 of a largest of at least 2^7. The scales are powers
# of two that differ by up to 2^spread within a tile, which costs the smallest as many bits.
P_ERROR = 2.0 ** -22
SHAPES = dict(SHAPES, hd64_g1=dict(qh=3, kvh=3, hd=64, ps=8), hd128_g16=dict(qh=16, kvh=1, hd=128, ps=16),
              hd256_g1=dict(qh=2, kvh=2, hd=256, ps=16))


def floor_of(w):
    return 2.0 ** (w.spread + 2 - 32)  # + 2: a row's largest element moves its scale as well


def gpu_decode(w, rule, out="fp32", opts=None, d=None, stream=None):
    t = torch()
    d = d or w.to_device()
    n = lib.pa_quant_workspace_size(w.prob(), opts)
    ws = t.full((max(n, 256),), 0xFF, dtype=t.uint8, device="cuda")  # NaN states: none is read
    o = t.full((w.batch, w.query_heads, w.head_dim), float("nan"), device="cuda",
               dtype=t.float16 if out == "fp16" else t.float32)
    lib.pa_decode_quant(w.prob(), device_rule(rule, out) if rule is not None else None, d["q"],
                        d["cache"], d["bt"], d["ctx"], w.scale, o, opts, ws if n else None, n,
                        stream=stream)
    t.cuda.synchronize()
    return o.cpu().numpy(), lib.pa_get_device_error()


def formula(w, rule):
    return attend(w, rule, P_ERROR, floor_of(w))


def check(w, rule, out="fp32", opts=None):
    got, flags = gpu_decode(w, rule, out, opts)
    assert flags == 0
    return assert_within(got, *formula(w, rule), out == "fp16")


@gpu
@pytest.mark.parametrize("rule", sorted(rules(QuantCached([1]))))
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_matches_formula(shape, rule):
    layout = len(shape + rule) % 2
    w = QuantCached(CTX, head_major=layout, q_scale=3.0, seed=1, **SHAPES[shape])
    check(w, rules(w)[rule], "fp16" if layout else "fp32")


OPTS = {
    "single": dict(schedule="single"),
    "balanced_few_workers": dict(schedule="balanced", workers=3),
    "balanced_many_workers": dict(schedule="balanced", workers=4000),
    "three_warps": dict(schedule="balanced", warps_per_cta=3),
    "one_warp": dict(schedule="single", warps_per_cta=1),
    "deep_ring": dict(schedule="balanced", stages=5, warps_per_cta=4),
    "no_ring": dict(schedule="single", stages=1),
}


@gpu
@pytest.mark.parametrize("opt", sorted(OPTS))
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_every_plan(shape, opt):
    w = QuantCached(CTX, q_scale=2.0, seed=2, **SHAPES[shape])
    check(w, rules(w)["all"], "fp32", lib.options(**OPTS[opt]))
    check(w, Rule(softcap=4.0), "fp16", lib.options(**OPTS[opt]))


@gpu
def test_rows_that_see_nothing_are_zero():
    w = QuantCached([5, 40, 1, 0, 90], **SHAPES["hd64_g2"])
    first = np.array([5, 1000, 1, 0, 89])  # past the query: nothing is seen; the last sees itself
    got, flags = gpu_decode(w, Rule(first=first))
    assert flags == 0 and (got[:4] == 0).all()
    last = w.gathered(4)[1][89].astype(np.float32)
    assert np.array_equal(got[4], np.repeat(last, 2, axis=0))  # one token: its value, exactly
    every = np.full(w.batch, 1 << 20)
    for opts in (None, lib.options(schedule="single")):
        got, flags = gpu_decode(w, Rule(first=every), opts=opts)
        assert flags == 0 and (got == 0).all()


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
@pytest.mark.parametrize("window", [1, 17, 64, 100])
def test_tokens_out_of_the_window_are_never_read(shape, window):
    """Their pages have left the table, their slots in a page that stays hold NaN codes and scales."""
    w = QuantCached([300, 64, 65, 129, 7], seed=4, **SHAPES[shape])
    rule = Rule(window=window, softcap=10.0)
    want = formula(w, rule)
    for b, n in enumerate(w.ctx):
        w.forget(b, max(0, int(n) - window))
    got, flags = gpu_decode(w, rule, "fp16")
    assert flags == 0
    assert_within(got, *want, True)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g1"])
def test_bits_do_not_depend_on_what_is_not_seen(shape):
    """Slots of no seen token, and scales that lie beside read ones, may hold anything."""
    w = QuantCached([75, 1, 130, 33], seed=5, **SHAPES[shape])
    outs = []
    for code, scale in ((0, 112), (0x7e, 135), (0x7f, 255), (0xff, 0), (0x7e, 254)):
        for name in "kv":
            unseen = ~np.isfinite(getattr(w, name)[..., 0])
            getattr(w, name + "_codes")[unseen] = code
            getattr(w, name + "_scales")[unseen] = scale
        got, flags = gpu_decode(w, Rule(softcap=20.0))
        assert flags == 0
        outs.append(got.view(np.uint32))
    for o in outs[1:]:
        assert np.array_equal(o, outs[0])


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_scales_of_the_whole_range(shape):
    """Scales from 2^-15 to 2^8, keys and values apart and mixed, in both orders along the context."""
    w = QuantCached([200, 47, 130], seed=6, q_scale=0.01, **SHAPES[shape])
    w.spread = 0
    for name, e in [("k", -15), ("k", 5), ("v", -15), ("v", 7)]:  # one exponent everywhere
        live = np.isfinite(getattr(w, name)[..., 0])
        getattr(w, name + "_scales")[live] = 127 + e
        redo(w)
        check(w, Rule())
    for order in (1, -1):  # values' exponents over the context
        for b in range(w.batch):
            n = int(w.ctx[b])
            for i, t in enumerate(range(n)[::order]):
                w.v_scales[w.bt[b, t // w.ps], t % w.ps] = 127 - 15 + 23 * i // n
        redo(w)
        w.spread = 23
        check(w, Rule())
        check(w, Rule(window=60))


def redo(w):
    """The numbers of codes and scales that a test has changed."""
    from tests.quant_reference import numbers

    for name in "kv":
        x = getattr(w, name)
        live = np.isfinite(x[..., 0])
        y = numbers(getattr(w, name + "_codes"), getattr(w, name + "_scales"))
        x[live] = y[live].astype(np.float16)
        assert (x[live].astype(np.float64) == y[live]).all()


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_largest_and_smallest_numbers(shape):
    """Rows of every code under the largest and smallest scale; sums of the largest values."""
    w = QuantCached([127, 40], seed=7, **SHAPES[shape])
    w.spread = 23
    rng = np.random.default_rng(8)
    for name in "kv":
        live = np.isfinite(getattr(w, name)[..., 0])
        c = rng.integers(0, 127, (int(live.sum()), w.head_dim)) | rng.choice([0, 128], (int(live.sum()), 1))
        e = rng.choice([-15, 8], int(live.sum()))
        c = np.where((e == 8)[:, None] & ((c & 127) > 119), 119, c)  # 240: what the format allows
        getattr(w, name + "_codes")[live] = c
        getattr(w, name + "_scales")[live] = e + 127
    redo(w)
    w.q = (w.q * 2.0 ** -14).astype(np.float16)
    check(w, Rule())
    check(w, Rule(softcap=2.0))
    w.q[:] = 0  # every token weighs the same
    check(w, Rule())


@gpu
def test_scores_far_past_the_cap_and_growing_maxima():
    w = QuantCached([500, 130], q_scale=40.0, seed=6, **SHAPES["hd128_g4"])
    check(w, Rule(softcap=30.0))
    for b in range(2):  # keys that grow along the sequence move the running maximum often
        for t in range(int(w.ctx[b])):
            w.k_scales[w.bt[b, t // w.ps], t % w.ps] = 127 - 9 + t // 60
    redo(w)
    check(w, Rule())
    check(w, Rule(softcap=200.0, slopes=-0.01 * slopes_of(w.query_heads)))
    w.scale = 0.0  # every seen token weighs the same
    check(w, Rule(window=70, softcap=3.0))
    check(w, Rule())
    w.scale = -0.05
    check(w, Rule(window=70, softcap=3.0))


@gpu
def test_biases_of_a_far_context():
    w = QuantCached([4096, 4000], seed=7, **SHAPES["hd64_g2"])
    check(w, Rule(slopes=np.array([1.0, 0.01, 1e-4, 30.0], dtype=np.float32)))


@gpu
def test_captured_replayed_and_two_graphs():
    """A captured call replays with other inputs in the same buffers, and two graphs with workspaces
    of their own do not disturb each other on two streams."""
    t = torch()
    w = QuantCached([700, 33, 2048], seed=8, **SHAPES["hd128_g4"])
    rule = Rule(softcap=5.0, window=1000)
    want = formula(w, rule)
    d, dr = w.to_device(), device_rule(rule, "fp32")
    n = lib.pa_quant_workspace_size(w.prob())
    graphs = []
    for _ in range(2):
        ws = t.empty(n, dtype=t.uint8, device="cuda")
        o = t.empty(w.batch, w.query_heads, w.head_dim, device="cuda")
        call = lambda: lib.pa_decode_quant(w.prob(), dr, d["q"], d["cache"], d["bt"], d["ctx"],  # noqa: E731
                                           w.scale, o, workspace=ws, workspace_bytes=n)
        call()
        t.cuda.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            call()
        graphs.append((g, ws, o, t.cuda.Stream()))
    first = None
    for _ in range(5):
        for _, _, o, _ in graphs:
            o.fill_(float("nan"))
        t.cuda.synchronize()
        for g, _, _, s in graphs:
            with t.cuda.stream(s):
                g.replay()
        t.cuda.synchronize()
        for _, _, o, _ in graphs:
            got = o.cpu().numpy()
            first = got if first is None else first
            assert np.array_equal(got, first)
    assert lib.pa_get_device_error() == 0
    assert_within(first, *want, False)
    w.q = (-w.q).astype(np.float16)
    d["q"].copy_(t.from_numpy(w.q))
    want = formula(w, rule)
    for g, _, o, _ in graphs:
        g.replay()
        t.cuda.synchronize()
        assert_within(o.cpu().numpy(), *want, False)


@gpu
def test_deterministic_and_codes_as_float8():
    t = torch()
    w = QuantCached([900, 33, 1500, 4], seed=10, **SHAPES["hd256_g6"])
    a, _ = gpu_decode(w, Rule(softcap=5.0))
    d = w.to_device()
    d["cache"] = lib.quant_cache(d["kc"].view(t.float8_e4m3fn), d["vc"].view(t.float8_e4m3fn),
                                 d["ks"], d["vs"])
    for _ in range(3):
        assert np.array_equal(gpu_decode(w, Rule(softcap=5.0), d=d)[0], a)


@gpu
def test_bad_pages_and_lengths_are_flagged():
    make = lambda: QuantCached([40, 60], maxp=8, **SHAPES["hd64_g2"])  # noqa: E731
    w = make()
    w.bt[1, 2] = w.pages
    got, flags = gpu_decode(w, Rule(softcap=5.0))
    assert flags == lib.PA_DEVERR_PAGE_ID
    assert_within(got[:1], *[x[:1] for x in formula(make(), Rule(softcap=5.0))], False)
    _, flags = gpu_decode(w, Rule(window=12))  # the bad page lies before the window: nobody reads it
    assert flags == 0
    w = make()
    w.ctx[0] = -1
    got, flags = gpu_decode(w, Rule())
    assert flags == lib.PA_DEVERR_CONTEXT and (got[0] == 0).all()
    full = QuantCached([128, 60], maxp=8, **SHAPES["hd64_g2"])  # too long: the table's capacity
    want = formula(full, Rule())
    full.ctx[0] = 129
    got, flags = gpu_decode(full, Rule())
    assert flags == lib.PA_DEVERR_CONTEXT
    assert_within(got, *want, False)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_expired_waits_are_reported_and_leave_the_next_call_alone(shape):
    w = QuantCached([900, 33], **SHAPES[shape])
    _, flags = gpu_decode(w, Rule(softcap=5.0), opts=lib.options(test_flags=lib.PA_TEST_EXPIRE_WAITS))
    assert flags == lib.PA_DEVERR_TIMEOUT
    check(w, Rule(softcap=5.0))


# ---------------------------------------------------------------------------- refusals
def decode(prob, score, args, **kw):
    return lib.status_of(lib.pa_decode_quant, prob, score, *args, **kw)


def test_refusals():
    prob = lib.problem(4, 32, 8, 128, 16, 256, 1024)
    cache = lib.quant_cache(GOOD, GOOD, GOOD, GOOD)
    args = [GOOD, cache, GOOD, GOOD, 0.1, GOOD]
    if not torch().cuda.is_available():
        assert decode(prob, lib.score(softcap=5.0), args) in (5, 6)
        assert decode(prob, None, args) in (5, 6)
    else:
        assert decode(prob, None, args) == 4  # no workspace
        n = lib.pa_quant_workspace_size(prob)
        assert decode(prob, None, args, workspace=GOOD, workspace_bytes=n - 1) == 4
        assert decode(prob, None, args, workspace=GOOD + 16, workspace_bytes=n) == 3
    for i, bad, status in [(0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (5, None, 1),
                           (4, float("nan"), 1), (4, float("inf"), 1), (0, GOOD + 8, 3),
                           (5, GOOD + 4, 3), (2, GOOD + 2, 3)]:
        a = list(args)
        a[i] = bad
        assert decode(prob, lib.score(), a) == status, (i, bad)
    for i in range(4):
        for bad, status in ((None, 1), (GOOD + 8, 3)):
            parts = [GOOD] * 4
            parts[i] = bad
            a = list(args)
            a[1] = lib.quant_cache(*parts)
            assert decode(prob, None, a) == status
    for kw, status in [(dict(softcap=-1.0), 1), (dict(softcap=float("nan")), 1), (dict(window=-1), 1),
                       (dict(out=2), 1), (dict(slopes=GOOD + 1), 3), (dict(first_tokens=GOOD + 2), 3)]:
        assert decode(prob, lib.score(**kw), args) == status, kw
    for o, status in [(dict(math="simt"), 2), (dict(combine="fused"), 2), (dict(schedule=7), 1),
                      (dict(tile_tokens=64), 2), (dict(stages=9), 1), (dict(stages=-1), 1),
                      (dict(warps_per_cta=9), 1), (dict(warps_per_cta=8, stages=8), 2)]:
        assert decode(prob, None, args, opts=lib.options(**o)) == status, o
    assert decode(lib.problem(4, 32, 8, 96, 16, 256, 1024), None, args) == 2
    assert decode(lib.problem(0, 32, 8, 128, 16, 256, 1024), None, args) == 0


def test_binding_refuses_tensors_it_cannot_pass():
    t = torch()
    prob = lib.problem(4, 4, 2, 64, 16, 256, 1024)
    cache = lib.quant_cache(GOOD, GOOD, GOOD, GOOD)
    args = [GOOD, cache, GOOD, GOOD, 0.1, GOOD]
    for i, x in [(0, t.zeros(4, 4, 64, dtype=t.float16)), (2, t.zeros(4, 256, dtype=t.int32))]:
        a = list(args)
        a[i] = x  # host memory
        assert decode(prob, None, a) == 1
    codes, scales = t.zeros(9, 16, 2, 64, dtype=t.uint8), t.zeros(9, 2, 16, dtype=t.uint8)
    with pytest.raises(lib.PagedAttnError):  # host memory
        lib.quant_cache(codes, codes, scales, scales)
    with pytest.raises(lib.PagedAttnError):  # not bytes
        lib.quant_cache(codes.to(t.float16), GOOD, GOOD, GOOD)
    with pytest.raises(lib.PagedAttnError):
        lib.norm(1e-6, t.ones(64))
