"""pa_decode_scored (a decode step with capped, biased and masked scores) against the formula in
64 bits, where it can go wrong; refusals on the host."""

import numpy as np
import pytest

from paged_kv_cache_63_gb300 import lib
from tests.gpu_util import torch
from tests.scored_reference import Cached, Rule, assert_within, attend, device_rule, slopes_of

gpu = pytest.mark.gpu
GOOD = 1 << 20

# 22 bits of a probability meet V (fp16 and its remainder in fp16); a weight is told from 0 down
# to 2^-25 against a largest of at least 2^7
P_ERROR, P_FLOOR = 2.0 ** -22, 2.0 ** -32


def gpu_decode(w, rule, out="fp32", opts=None, d=None, stream=None):
    t = torch()
    d = d or w.to_device()
    n = lib.pa_workspace_size(w.prob(), opts)
    ws = t.full((max(n, 256),), 0xFF, dtype=t.uint8, device="cuda")  # NaN states: none is read
    o = t.full((w.batch, w.query_heads, w.head_dim), float("nan"), device="cuda",
               dtype=t.float16 if out == "fp16" else t.float32)
    lib.pa_decode_scored(w.prob(), device_rule(rule, out) if rule is not None else None, d["q"],
                         d["k"], d["v"], d["bt"], d["ctx"], w.scale, o, opts, ws if n else None, n,
                         stream=stream)
    t.cuda.synchronize()
    return o.cpu().numpy(), lib.pa_get_device_error()


def check(w, rule, out="fp32", opts=None):
    got, flags = gpu_decode(w, rule, out, opts)
    assert flags == 0
    return assert_within(got, *attend(w, rule, P_ERROR, P_FLOOR), out == "fp16")


CTX = [1, 2, 15, 16, 17, 33, 64, 100, 257, 0, 700]
SHAPES = {
    "hd64_g2": dict(qh=4, kvh=2, hd=64, ps=16),
    "hd128_g4": dict(qh=32, kvh=8, hd=128, ps=16),
    "hd128_g1": dict(qh=4, kvh=4, hd=128, ps=8),
    "hd256_g6": dict(qh=12, kvh=2, hd=256, ps=64),
    "hd64_g12": dict(qh=12, kvh=1, hd=64, ps=32),  # two units a K/V head
    "hd128_g5": dict(qh=15, kvh=3, hd=128, ps=256),
}


def rules(w):
    b, qh = w.batch, w.query_heads
    first = np.minimum(np.arange(b) * 5, np.maximum(w.ctx - 1, 0))
    return {
        "none": Rule(),
        "cap": Rule(softcap=2.0),
        "window1": Rule(window=1),
        "window16": Rule(window=16),
        "window21": Rule(window=21),
        "window_long": Rule(window=1 << 30),
        "slopes": Rule(slopes=slopes_of(qh)),
        "first": Rule(first=first),
        "all": Rule(softcap=3.0, window=90, slopes=slopes_of(qh), first=first),
    }


@gpu
@pytest.mark.parametrize("rule", sorted(rules(Cached([1]))))
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_matches_formula(shape, rule):
    layout = len(shape + rule) % 2
    w = Cached(CTX, head_major=layout, q_scale=3.0, seed=1, **SHAPES[shape])
    check(w, rules(w)[rule], "fp16" if layout else "fp32")


OPTS = {
    "single": dict(schedule="single"),
    "balanced_few_workers": dict(schedule="balanced", workers=3),
    "balanced_many_workers": dict(schedule="balanced", workers=4000),
    "two_stages": dict(schedule="balanced", stages=2, warps_per_cta=4),
    "tile32": dict(tile_tokens=32),
}


@gpu
@pytest.mark.parametrize("opt", sorted(OPTS))
def test_every_plan(opt):
    w = Cached(CTX, q_scale=2.0, seed=2, **SHAPES["hd128_g4"])
    rule = rules(w)["all"]
    check(w, rule, "fp32", lib.options(**OPTS[opt]))
    check(w, Rule(softcap=4.0), "fp16", lib.options(**OPTS[opt]))


@gpu
def test_rows_that_see_nothing_are_zero():
    w = Cached([5, 40, 1, 0, 90], **SHAPES["hd64_g2"])
    first = np.array([5, 1000, 1, 0, 89])  # past the query: nothing is seen; the last sees itself
    got, flags = gpu_decode(w, Rule(first=first))
    assert flags == 0
    assert (got[:4] == 0).all()
    last = w.gathered(4)[1][89].astype(np.float32)
    assert np.array_equal(got[4], np.repeat(last, 2, axis=0))  # one token: its value, exactly
    every = np.full(w.batch, 1 << 20)
    for opts in (None, lib.options(schedule="single")):
        got, flags = gpu_decode(w, Rule(first=every), opts=opts)
        assert flags == 0 and (got == 0).all()


@gpu
def test_negative_first_tokens_mean_zero_and_prefixes_change_nothing():
    w = Cached([30, 200], **SHAPES["hd128_g4"])
    a, _ = gpu_decode(w, Rule(softcap=5.0))
    b, _ = gpu_decode(w, Rule(softcap=5.0, first=np.array([-3, -(1 << 31)]),
                              prefix=np.array([10, 500])))
    assert np.array_equal(a, b)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
@pytest.mark.parametrize("window", [1, 17, 64, 100])
def test_tokens_out_of_the_window_are_never_read(shape, window):
    """Their pages have left the table, their slots in a page that stays hold NaN and Inf."""
    w = Cached([300, 64, 65, 129, 7], seed=4, **SHAPES[shape])
    rule = Rule(window=window, softcap=10.0)
    want = attend(w, rule, P_ERROR, P_FLOOR)
    for b, n in enumerate(w.ctx):
        w.forget(b, max(0, int(n) - window))
    got, flags = gpu_decode(w, rule, "fp16")
    assert flags == 0
    assert_within(got, *want, True)


@gpu
def test_scores_far_past_the_cap_and_growing_maxima():
    w = Cached([500, 130], q_scale=40.0, seed=6, **SHAPES["hd128_g4"])
    check(w, Rule(softcap=30.0))
    for b in range(2):  # keys that grow along the sequence move the running maximum often
        for t in range(int(w.ctx[b])):
            page, slot = w.bt[b, t // w.ps], t % w.ps
            w.k[page, slot] = (w.k[page, slot].astype(np.float32) * (1 + t / 40)).astype(np.float16)
    check(w, Rule())
    check(w, Rule(softcap=200.0, slopes=-0.01 * slopes_of(w.query_heads)))
    w.scale = 0.0  # every seen token weighs the same
    check(w, Rule(window=70, softcap=3.0))
    check(w, Rule())
    w.scale = -0.05
    check(w, Rule(window=70, softcap=3.0))


@gpu
def test_biases_of_a_far_context():
    """4096 tokens under steep and shallow slopes; distances far past what the softmax keeps."""
    w = Cached([4096, 4000], seed=7, **SHAPES["hd64_g2"])
    check(w, Rule(slopes=np.array([1.0, 0.01, 1e-4, 30.0], dtype=np.float32)))


@gpu
def test_captured_and_replayed():
    """A captured call replays with other inputs in the same buffers, as often as one likes, and
    two graphs with workspaces of their own do not disturb each other."""
    t = torch()
    w = Cached([700, 33, 2048], seed=8, **SHAPES["hd128_g4"])
    rule = Rule(softcap=5.0, window=1000)
    want = attend(w, rule, P_ERROR, P_FLOOR)
    d, dr = w.to_device(), device_rule(rule, "fp32")
    n = lib.pa_workspace_size(w.prob())
    graphs = []
    for _ in range(2):
        ws = t.empty(n, dtype=t.uint8, device="cuda")
        o = t.empty(w.batch, w.query_heads, w.head_dim, device="cuda")
        call = lambda: lib.pa_decode_scored(w.prob(), dr, d["q"], d["k"], d["v"], d["bt"],  # noqa: E731
                                            d["ctx"], w.scale, o, workspace=ws, workspace_bytes=n)
        call()
        t.cuda.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            call()
        graphs.append((g, ws, o))
    first = None
    for _ in range(5):
        for g, _, o in graphs:
            o.fill_(float("nan"))
            g.replay()
        t.cuda.synchronize()
        for _, _, o in graphs:
            got = o.cpu().numpy()
            first = got if first is None else first
            assert np.array_equal(got, first)
    assert_within(first, *want, False)
    w.q = (-w.q).astype(np.float16)
    d["q"].copy_(t.from_numpy(w.q))
    want = attend(w, rule, P_ERROR, P_FLOOR)
    for g, _, o in graphs:
        g.replay()
        t.cuda.synchronize()
        assert_within(o.cpu().numpy(), *want, False)


@gpu
def test_on_another_stream_and_two_calls_at_once():
    t = torch()
    w = Cached([900, 33, 1500], seed=9, **SHAPES["hd128_g4"])
    rule = Rule(softcap=5.0)
    want = attend(w, rule, P_ERROR, P_FLOOR)
    d, dr = w.to_device(), device_rule(rule, "fp16")
    n = lib.pa_workspace_size(w.prob())
    t.cuda.synchronize()
    made = []
    for _ in range(2):
        s = t.cuda.Stream()
        ws = t.empty(n, dtype=t.uint8, device="cuda")
        o = t.empty(w.batch, w.query_heads, w.head_dim, device="cuda", dtype=t.float16)
        made.append((s, ws, o))
    t.cuda.synchronize()
    for _ in range(10):
        for s, ws, o in made:
            lib.pa_decode_scored(w.prob(), dr, d["q"], d["k"], d["v"], d["bt"], d["ctx"], w.scale, o,
                                 workspace=ws, workspace_bytes=n, stream=s)
    t.cuda.synchronize()
    for _, _, o in made:
        assert_within(o.cpu().numpy(), *want, True)


@gpu
def test_deterministic():
    w = Cached([900, 33, 1500, 4], seed=10, **SHAPES["hd256_g6"])
    a, _ = gpu_decode(w, Rule(softcap=5.0))
    for _ in range(3):
        assert np.array_equal(gpu_decode(w, Rule(softcap=5.0))[0], a)


@gpu
def test_bad_pages_and_lengths_are_flagged():
    w = Cached([40, 60], maxp=8, **SHAPES["hd64_g2"])
    w.bt[1, 2] = w.pages
    got, flags = gpu_decode(w, Rule(softcap=5.0))
    assert flags == lib.PA_DEVERR_PAGE_ID
    assert_within(got[:1], *[x[:1] for x in attend(Cached([40, 60], maxp=8, **SHAPES["hd64_g2"]),
                                                   Rule(softcap=5.0), P_ERROR, P_FLOOR)], False)
    # the bad page lies before the window: nobody reads it
    _, flags = gpu_decode(w, Rule(window=12))
    assert flags == 0
    w = Cached([40, 60], maxp=8, **SHAPES["hd64_g2"])
    w.ctx[0] = -1
    got, flags = gpu_decode(w, Rule())
    assert flags == lib.PA_DEVERR_CONTEXT and (got[0] == 0).all()


@gpu
def test_expired_waits_are_reported_and_leave_the_next_call_alone():
    w = Cached([900, 33], **SHAPES["hd128_g4"])
    _, flags = gpu_decode(w, Rule(softcap=5.0), opts=lib.options(test_flags=lib.PA_TEST_EXPIRE_WAITS))
    assert flags == lib.PA_DEVERR_TIMEOUT
    check(w, Rule(softcap=5.0))


def decode(prob, score, args, **kw):
    return lib.status_of(lib.pa_decode_scored, prob, score, *args, **kw)


def test_refusals():
    prob = lib.problem(4, 32, 8, 128, 16, 256, 1024)
    args = [GOOD, GOOD, GOOD, GOOD, GOOD, 0.1, GOOD]
    on_gpu = torch().cuda.is_available()
    if not on_gpu:
        assert decode(prob, lib.score(softcap=5.0), args) in (5, 6)
        assert decode(prob, None, args) in (5, 6)
    else:
        assert decode(prob, None, args) == 4  # no workspace
        n = lib.pa_workspace_size(prob)
        assert decode(prob, None, args, workspace=GOOD, workspace_bytes=n - 1) == 4
        assert decode(prob, None, args, workspace=GOOD + 16, workspace_bytes=n) == 3
    for i, bad, status in [(0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (4, None, 1),
                           (6, None, 1), (5, float("nan"), 1), (5, float("inf"), 1),
                           (0, GOOD + 8, 3), (6, GOOD + 4, 3), (3, GOOD + 2, 3)]:
        a = list(args)
        a[i] = bad
        assert decode(prob, lib.score(), a) == status, (i, bad)
    for kw, status in [(dict(softcap=-1.0), 1), (dict(softcap=float("nan")), 1),
                       (dict(softcap=float("inf")), 1), (dict(softcap=1e-45), 1),
                       (dict(softcap=3e38), 1), (dict(window=-1), 1), (dict(out=2), 1),
                       (dict(out=-1), 1), (dict(slopes=GOOD + 1), 3),
                       (dict(first_tokens=GOOD + 2), 3), (dict(prefix_lengths=GOOD + 3), 3)]:
        assert decode(prob, lib.score(**kw), args) == status, kw
    s = lib.score()
    s.reserved = 1
    assert decode(prob, s, args) == 1
    for o, status in [(dict(math="simt"), 2), (dict(combine="fused"), 2), (dict(schedule=7), 1),
                      (dict(tile_tokens=64), 2)]:
        assert decode(prob, None, args, opts=lib.options(**o)) == status, o
    assert decode(lib.problem(4, 32, 8, 96, 16, 256, 1024), None, args) == 2
    assert decode(lib.problem(0, 32, 8, 128, 16, 256, 1024), None, args) == 0


def test_binding_refuses_tensors_it_cannot_pass():
    t = torch()
    prob = lib.problem(4, 4, 2, 64, 16, 256, 1024)
    args = [GOOD, GOOD, GOOD, GOOD, GOOD, 0.1, GOOD]
    for i, x in [(0, t.zeros(4, 4, 64, dtype=t.float16)), (3, t.zeros(4, 256, dtype=t.int32))]:
        a = list(args)
        a[i] = x  # host memory
        assert decode(prob, None, a) == 1
    with pytest.raises(lib.PagedAttnError):
        lib.score(slopes=t.zeros(4))
