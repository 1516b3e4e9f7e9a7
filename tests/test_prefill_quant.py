"""pa_prefill_quant (several new tokens per sequence over a quantised cache) against the formula in 64
bits and against pa_prefill_scored over the numbers that the codes stand for, bit for bit; refusals on
the host; a layer's run over a quantised cache; caches of more than 2^31 elements."""

import numpy as np
import pytest

from paged_kv_cache_63_gb300 import lib
from tests.gpu_util import torch
from tests.quant_reference import QuantCached, numbers
from tests.scored_reference import Rule, assert_within, attend, device_rule, slopes_of
from tests.test_prefill_scored import CTX, ERRORS, NEW, SHAPES, documents, rules

gpu = pytest.mark.gpu
GOOD = 1 << 20
SHAPES = dict(SHAPES, hd64_g1=dict(qh=2, kvh=2, hd=64, ps=8), hd256_page16=dict(qh=4, kvh=2, hd=256, ps=16),
              hd128_page64=dict(qh=8, kvh=2, hd=128, ps=64))


def case(shape, seed=1, **kw):
    args = dict(ctx=CTX, new=NEW, q_scale=3.0, seed=seed, pad=3)
    args.update(SHAPES[shape])
    args.update(kw)
    return QuantCached(args.pop("ctx"), args.pop("new"), **args)


def gpu_prefill(w, rule, opts=None, d=None, max_query_len=None, stream=None, codes=True):
    t = torch()
    d = d or w.to_device()
    o = t.full((w.rows, w.query_heads, w.head_dim), float("nan"), device="cuda", dtype=t.float16)
    most = int(w.new.max()) if max_query_len is None else max_query_len
    if codes:
        lib.pa_prefill_quant(w.prob(), device_rule(rule, "fp16"), d["q"], d["qs"], w.rows, most,
                             d["cache"], d["bt"], d["ctx"], w.scale, o, opts, stream=stream)
    else:
        lib.pa_prefill_scored(w.prob(), device_rule(rule, "fp16"), d["q"], d["qs"], w.rows, most,
                              d["k"], d["v"], d["bt"], d["ctx"], w.scale, o, opts, stream=stream)
    t.cuda.synchronize()
    return o.cpu().numpy(), lib.pa_get_device_error()


def few(w, rule, most):
    """Whether the call goes to the kernel for few rows (tests/test_prefill_few_quant.py)."""
    rows = most * (w.query_heads // w.kv_heads)
    sms = torch().cuda.get_device_properties(0).multi_processor_count
    ctas, items = (-(-rows // n) * w.kv_heads * w.batch for n in (8, 128))
    return rule.first is None and ctas <= 2 * max(sms, items)


def check(w, rule, **kw):
    """Within the formula's bound, and (but for few rows) the bits of the call over the numbers
    themselves."""
    d = w.to_device()
    got, flags = gpu_prefill(w, rule, d=d, **kw)
    assert flags == 0
    want, bound = attend(w, rule, **ERRORS)
    assert np.isnan(got[np.isnan(want)]).all()  # rows of no new token are left alone
    assert_within(got, want, bound, True)
    if few(w, rule, kw.get("max_query_len") or int(w.new.max())):
        return  # the kernel for few rows, whose sums are in another order
    plain, flags = gpu_prefill(w, rule, d=d, codes=False, **kw)
    assert flags == 0
    assert np.array_equal(got.view(np.uint16), plain.view(np.uint16))


@gpu
@pytest.mark.parametrize("rule", sorted(rules(case("hd64_g2"))))
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_matches_formula(shape, rule):
    w = case(shape, head_major=len(shape + rule) % 2)
    check(w, rules(w)[rule])


@gpu
@pytest.mark.parametrize("pad", [0, 2])
def test_no_new_tokens(pad):
    w = case("hd128_g4", ctx=[40, 0], new=[0, 0], pad=pad)
    check(w, Rule(softcap=3.0), max_query_len=1)


@gpu
@pytest.mark.parametrize("parts", range(8))
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g6", "hd256_g6"])
def test_every_kernel_of_a_rule(shape, parts):
    w = case(shape, ctx=[150, 70, 3], new=[150, 20, 3], seed=parts)
    rule = dict(softcap=4.0 if parts & 1 else 0.0,
                slopes=slopes_of(w.query_heads) if parts & 2 else None,
                first=documents(w, 25) if parts & 4 else None)
    check(w, Rule(**rule), max_query_len=2500)  # (a grid for many rows)
    check(w, Rule(window=40, prefix=np.array([90, 0, 2]), **rule), max_query_len=2500)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g1", "hd256_g1"])
def test_one_new_token_each(shape):
    w = case(shape, ctx=[1, 2, 128, 129, 400, 257], new=[1] * 6)
    for rule in (Rule(softcap=5.0), Rule(window=130), Rule(first=np.array([0, 1, 127, 128, 3, 250, 0, 0, 0]))):
        check(w, rule)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_rows_that_see_nothing_are_zero(shape):
    w = case(shape)
    first = np.zeros(w.rows, dtype=np.int64)
    first[:140] = 1 << 20        # the first sequence's first tiles
    first[150:151] = 10000
    first[301:] = np.arange(w.rows - 301) * 7  # some of them past their query
    check(w, Rule(first=first))
    check(w, Rule(first=np.full(w.rows, 1 << 30), softcap=4.0))


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
@pytest.mark.parametrize("window", [1, 33, 128, 200])
def test_tokens_nobody_sees_are_never_read(shape, window):
    w = case(shape, ctx=[700, 411, 129], new=[90, 1, 129], pad=0)
    rule = Rule(window=window, softcap=10.0)
    want = attend(w, rule, **ERRORS)
    for b in range(w.batch):
        w.forget(b, max(0, int(w.ctx[b] - w.new[b]) - window + 1))
    got, flags = gpu_prefill(w, rule)
    assert flags == 0
    assert_within(got, *want, True)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd128_g6", "hd256_g6", "hd256_g1"])
def test_tokens_nobody_sees_between_seen_ones(shape):
    """Rows that see nothing leave their own tokens unseen between tokens that other rows see: those
    hold NaN codes and scales, and pages of nothing else have left the table."""
    w = case(shape, ctx=[700, 411], new=[200, 150], pad=0)
    first = np.zeros(w.rows, dtype=np.int64)
    never = 1 << 30
    first[5:40] = never
    first[40:150] = 540 + np.arange(110) // 2
    first[150:195] = never
    first[195:200] = 699
    for j in range(150):
        first[200 + j] = 411 - 150 + j if j % 3 == 0 else never
    rule = Rule(first=first, softcap=10.0)
    want = attend(w, rule, **ERRORS)
    for b in range(w.batch):
        n = int(w.ctx[b])
        seen = np.zeros(n + w.ps, dtype=bool)
        for row, pos in w.rows_of(b):
            seen[first[row]:pos + 1] = True
        for t in range(n):
            if not seen[t]:
                at = w.bt[b, t // w.ps], t % w.ps
                w.k_codes[at], w.k_scales[at] = 0x7f, 255
                w.v_codes[at], w.v_scales[at] = 0xff, 254
        for page in range(-(-n // w.ps)):
            if not seen[page * w.ps:(page + 1) * w.ps].any():
                w.bt[b, page] = -5
    got, flags = gpu_prefill(w, rule)
    assert flags == 0
    assert_within(got, *want, True)


@gpu
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd128_g6", "hd256_g6"])
def test_bits_do_not_depend_on_what_is_not_seen(shape, slopes):
    """Slots outside the contexts, tokens before the window and rows of no new token may hold large
    numbers, which would take another form of tanh, or NaN."""
    w = case(shape, ctx=[300, 1, 129, 200], new=[170, 1, 60, 31], q_scale=1.0, pad=5)
    rule = Rule(softcap=20.0, window=100, slopes=slopes_of(w.query_heads) if slopes else None)
    for b in range(w.batch):
        w.forget(b, max(0, int(w.ctx[b] - w.new[b]) - rule.window + 1))
    rows = int(w.qs[-1])
    unseen = {x: ~np.isfinite(getattr(w, x)[..., 0]) for x in "kv"}
    outs = []
    for fill, code, scale in ((0.0, 0, 127), (3000.0, 0x7e, 135), (np.nan, 0x7f, 255), (1.0, 0x7e, 0)):
        for x in "kv":
            getattr(w, x + "_codes")[unseen[x]] = code
            getattr(w, x + "_scales")[unseen[x]] = scale
        w.q[rows:] = fill
        out, flags = gpu_prefill(w, rule)
        assert flags == 0
        outs.append(out[:rows].view(np.uint16))
    for o in outs[1:]:
        assert np.array_equal(outs[0], o)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_scales_of_the_whole_range_and_growing_maxima(shape):
    w = case(shape, ctx=[600, 300], new=[500, 300], pad=0)
    for b in range(w.batch):
        n = int(w.ctx[b])
        for t in range(n):
            at = w.bt[b, t // w.ps], t % w.ps
            w.k_scales[at] = 127 - 15 + 9 * t // n
            w.v_scales[at] = 127 - 15 + 23 * ((t * 7) % n) // n
    for x in "kv":
        live = np.isfinite(getattr(w, x)[..., 0])
        y = numbers(getattr(w, x + "_codes"), getattr(w, x + "_scales"))
        big = np.abs(y[live]).max(-1) > 61440  # keep to what the format allows
        at = tuple(i[big] for i in np.nonzero(live))
        getattr(w, x + "_codes")[at] &= 0xbf
        y = numbers(getattr(w, x + "_codes"), getattr(w, x + "_scales"))
        getattr(w, x)[live] = y[live].astype(np.float16)
        assert (getattr(w, x)[live].astype(np.float64) == y[live]).all()
    check(w, Rule())
    check(w, Rule(softcap=20.0))
    check(w, Rule(softcap=500.0, window=250))
    check(w, Rule(slopes=-0.05 * slopes_of(w.query_heads), first=documents(w, 150)))


@gpu
def test_negative_scale_and_steep_biases():
    w = case("hd128_g4")
    assert not few(w, Rule(), 300)
    w.scale = -w.scale
    check(w, Rule())
    check(w, Rule(softcap=6.0, slopes=100.0 * slopes_of(w.query_heads)))
    w.scale = 0.0  # every seen token weighs the same
    check(w, Rule(window=70))
    check(w, Rule(slopes=slopes_of(w.query_heads)))


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_grid_taller_than_needed(shape):
    w = case(shape)
    check(w, Rule(softcap=9.0, prefix=w.ctx), max_query_len=900)


@gpu
@pytest.mark.parametrize("shape", ["hd128_g4", "hd256_g6"])
def test_more_items_than_sms_deterministic_and_replayed(shape):
    t = torch()
    b = 40
    ctx = np.arange(b) * 9 % 500 + 130
    w = case(shape, ctx=ctx, new=ctx - 1, pad=0)
    rule = Rule(softcap=8.0, window=200, first=documents(w, 200))
    want = attend(w, rule, **ERRORS)
    d, dr = w.to_device(), device_rule(rule, "fp16")
    o = t.zeros(w.rows, w.query_heads, w.head_dim, device="cuda", dtype=t.float16)
    call = lambda: lib.pa_prefill_quant(  # noqa: E731
        w.prob(), dr, d["q"], d["qs"], w.rows, int(w.new.max()), d["cache"], d["bt"], d["ctx"],
        w.scale, o)
    call()
    t.cuda.synchronize()
    first = o.cpu().numpy()
    assert lib.pa_get_device_error() == 0
    assert_within(first, *want, True)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        call()
    for _ in range(3):
        o.fill_(float("nan"))
        g.replay()
        t.cuda.synchronize()
        assert np.array_equal(o.cpu().numpy(), first)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g1", "hd256_g6", "hd256_g1"])
@pytest.mark.parametrize("window", [1, 40, 150])
def test_many_short_items(shape, window):
    b = 300
    ctx = np.arange(b) * 37 % 230 + 20
    w = case(shape, ctx=ctx, new=np.minimum(ctx, 20 + np.arange(b) % 60), pad=0)
    rule = Rule(window=window, softcap=9.0)
    want = attend(w, rule, **ERRORS)
    d, first = w.to_device(), None
    for _ in range(8):
        got, flags = gpu_prefill(w, rule, d=d)
        assert flags == 0
        first = got if first is None else first
        assert np.array_equal(got, first)
    assert_within(first, *want, True)


@gpu
def test_two_calls_at_once():
    t = torch()
    w = case("hd128_g4")
    rule = Rule(softcap=8.0, window=100)
    want = attend(w, rule, **ERRORS)
    d, dr = w.to_device(), device_rule(rule, "fp16")
    outs = [t.zeros(w.rows, 8, 128, device="cuda", dtype=t.float16) for _ in range(2)]
    streams = [t.cuda.Stream() for _ in range(2)]
    t.cuda.synchronize()
    for _ in range(5):
        for o, s in zip(outs, streams):
            lib.pa_prefill_quant(w.prob(), dr, d["q"], d["qs"], w.rows, 300, d["cache"], d["bt"],
                                 d["ctx"], w.scale, o, stream=s)
    t.cuda.synchronize()
    live = ~np.isnan(want[0])
    for o in outs:
        assert_within(o.cpu().numpy(), want[0], want[1], True)
        assert (o.cpu().numpy()[~live] == 0).all()


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_bad_offsets_lengths_and_pages_are_flagged(shape):
    w = case(shape)
    d, rule = w.to_device(), Rule(window=150)
    t = torch()
    for name, value, flag in [("ctx", [300, 1, 129, -1, 0, 77], lib.PA_DEVERR_CONTEXT),
                              ("ctx", [300, 1, 59, 200, 0, 77], lib.PA_DEVERR_QUERY_START),
                              ("qs", [0, 300, 301, 361, 361, 361, 9999], lib.PA_DEVERR_QUERY_START)]:
        bad = dict(d, **{name: t.tensor(value, dtype=t.int32, device="cuda")})
        _, flags = gpu_prefill(w, rule, d=bad)
        assert flags == flag
    w.bt[0, 0] = w.pages
    want = attend(case(shape), rule, **ERRORS)
    got, flags = gpu_prefill(w, rule)
    assert flags == lib.PA_DEVERR_PAGE_ID
    other = slice(int(w.qs[1]), int(w.qs[-1]))  # the other sequences' rows are unharmed
    assert_within(got[other], want[0][other], want[1][other], True)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_expired_wait_is_reported(shape):
    w = case(shape)
    _, flags = gpu_prefill(w, Rule(softcap=5.0), lib.options(test_flags=lib.PA_TEST_EXPIRE_WAITS))
    assert flags & lib.PA_DEVERR_TIMEOUT
    check(w, Rule(softcap=5.0))


# ---------------------------------------------------------------------------- a layer's run
@gpu
@pytest.mark.parametrize("head_major", [0, 1])
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_append_prefill_decode_and_read_together(shape, head_major):
    """As a serving loop runs a layer over a quantised cache: prompts normed, turned, appended and
    attended, then decode steps, each an append of one token and a decode; at the end the rows are
    read back. Every output is checked against the formula over the cache the calls wrote, and the
    cache against the format."""
    from tests.test_decode_quant import P_ERROR
    from tests.test_quant_cache import QuantCase

    t = torch()
    steps, lens = 4, np.array([130, 5, 64])
    s = dict(SHAPES[shape], head_major=head_major)
    qh, kvh, hd = s["qh"], s["kvh"], s["hd"]
    whole = QuantCase(lens + steps, lens + steps, seed=4, **s)  # the whole run as one append
    d = whole.put()
    codes = lib.quant_cache(d["k"], d["v"], d["ks"], d["vs"])
    norm = lib.norm(1e-6, d["q_weight"], d["k_weight"])
    rope = lib.rope(hd, "half", d["table"])
    prob, rule = whole.prob(), Rule(softcap=12.0, window=60)
    n_ws = lib.pa_quant_workspace_size(prob)
    ws = t.empty(max(n_ws, 256), dtype=t.uint8, device="cuda")
    put = lambda x: t.from_numpy(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
    w = QuantCached(lens + steps, np.zeros(3, dtype=int), **s)  # the formula's view
    w.bt, w.pages, w.maxp = whole.bt, whole.pages, whole.maxp
    for step in range(steps + 1):
        new = lens if step == 0 else np.ones(3, dtype=int)
        ctx = lens + step
        rows = np.concatenate([whole.qs[b] + np.arange(ctx[b] - new[b], ctx[b]) for b in range(3)])
        qkv = d["qkv"][t.from_numpy(rows).cuda()].contiguous()
        qs = np.concatenate([[0], np.cumsum(new)])
        q = t.empty(len(rows), qh, hd, dtype=t.float16, device="cuda")
        o = t.empty_like(q)
        lib.pa_append_quant(prob, norm, rope, qkv[:, :qh], qkv[:, qh:qh + kvh], qkv[:, qh + kvh:],
                            put(qs), len(rows), d["bt"], put(ctx), q, codes)
        dr = device_rule(rule, "fp16")
        if step == 0:
            lib.pa_prefill_quant(prob, dr, q, put(qs), len(rows), int(new.max()), codes, d["bt"],
                                 put(ctx), w.scale, o)
        else:
            lib.pa_decode_quant(prob, dr, q, codes, d["bt"], put(ctx), w.scale, o, workspace=ws,
                                workspace_bytes=n_ws)
        (_, got, scales), flags = whole.results(d)
        assert flags == 0
        w.ctx, w.new, w.rows, w.qs = ctx.astype(np.int32), new, len(rows), qs
        w.q, w.k, w.v = q.cpu().numpy(), numbers(got["k"], scales["k"]), numbers(got["v"], scales["v"])
        if step == 0:
            assert_within(o.cpu().numpy(), *attend(w, rule, **ERRORS), True)
        else:  # scales of a few powers of two: at most 7 bits from the smallest row to the largest
            assert_within(o.cpu().numpy(), *attend(w, rule, P_ERROR, 2.0 ** -25), True)
        want, tol, _, _ = whole.expected()
        assert (np.abs(w.q - want[rows]) <= tol[rows]).all()
    _, _, want_codes, want_scales = whole.expected()
    k, v = (t.empty(whole.total, kvh, hd, dtype=t.float16, device="cuda") for _ in range(2))
    lib.pa_read_quant(prob, codes, d["qs"], whole.total, d["bt"], d["ctx"], k, v)
    t.cuda.synchronize()
    assert lib.pa_get_device_error() == 0
    for x, read in (("k", k), ("v", v)):
        assert np.array_equal(scales[x], want_scales[x])
        assert np.array_equal(numbers(got[x], scales[x]), numbers(want_codes[x], scales[x]))
        for b in range(3):
            at = np.arange(lens[b] + steps)
            rows = numbers(got[x], scales[x])[whole.bt[b, at // whole.ps], at % whole.ps]
            assert np.array_equal(read[whole.qs[b]:whole.qs[b + 1]].cpu().numpy(), rows)


@gpu
@pytest.mark.parametrize("head_major", [0, 1])
def test_pages_past_32_bit_offsets(head_major):
    """Appended to, read and attended from pages that lie more than 2^32 bytes into the caches: the
    same bits as from a small cache."""
    t = torch()
    qh, kvh, hd, ps = 16, 8, 256, 256
    ctx, rows = [400, 300], 700
    far = 8400  # pages of 2^19 bytes
    g = t.Generator(device="cuda").manual_seed(5)
    qkv = t.randn(rows, qh + 2 * kvh, hd, generator=g, device="cuda", dtype=t.float16)
    ang = t.rand(512, 32, generator=g, device="cuda") * 6
    rope = lib.rope(64, "interleaved", t.stack([ang.cos(), ang.sin()], 1).contiguous())
    put = lambda x: t.tensor(x, dtype=t.int32, device="cuda")  # noqa: E731
    qs, dctx = put([0, 400, 700]), put(ctx)
    shape = (kvh, ps, hd) if head_major else (ps, kvh, hd)
    outs = []
    for pages, table in [(4, [[2, 0], [3, 1]]), (far, [[far - 1, 4097], [4, 8193]])]:
        k, v = (t.full((pages, *shape), 0x7f, dtype=t.uint8, device="cuda") for _ in range(2))
        ks, vs = (t.full((pages, kvh, ps), 255, dtype=t.uint8, device="cuda") for _ in range(2))
        codes, bt = lib.quant_cache(k, v, ks, vs), put(table)
        prob = lib.problem(2, qh, kvh, hd, ps, 2, pages, head_major)
        q = t.empty(rows, qh, hd, dtype=t.float16, device="cuda")
        o, last = t.empty_like(q), t.empty(2, qh, hd, dtype=t.float16, device="cuda")
        rk, rv = (t.empty(rows, kvh, hd, dtype=t.float16, device="cuda") for _ in range(2))
        rule = lib.score(softcap=20.0, window=150, out="fp16")
        lib.pa_append_quant(prob, None, rope, qkv[:, :qh], qkv[:, qh:qh + kvh], qkv[:, qh + kvh:], qs,
                            rows, bt, dctx, q, codes)
        lib.pa_prefill_quant(prob, rule, q, qs, rows, 400, codes, bt, dctx, 0.0625, o)
        n = lib.pa_quant_workspace_size(prob)
        ws = t.empty(max(n, 256), dtype=t.uint8, device="cuda")
        lib.pa_decode_quant(prob, rule, q[[399, 699]].contiguous(), codes, bt, dctx, 0.0625, last,
                            workspace=ws, workspace_bytes=n)
        lib.pa_read_quant(prob, codes, qs, rows, bt, dctx, rk, rv)
        t.cuda.synchronize()
        assert lib.pa_get_device_error() == 0
        outs.append([x.cpu().numpy() for x in (q, o, last, rk, rv)])
        assert int((ks != 255).sum()) == rows * kvh  # nothing else was written
        del k, v, ks, vs
        t.cuda.empty_cache()
    for small, large in zip(*outs):
        assert np.isfinite(small).all()
        assert np.array_equal(small.view(np.uint16), large.view(np.uint16))


# ---------------------------------------------------------------------------- refusals
def prefill(prob, score, a, **kw):
    return lib.status_of(lib.pa_prefill_quant, prob, score, *a, **kw)


def test_refusals():
    prob = lib.problem(4, 32, 8, 128, 16, 256, 1024)
    half = lib.score(softcap=5.0, out="fp16")
    cache = lib.quant_cache(GOOD, GOOD, GOOD, GOOD)
    # query, query_start, total_tokens, max_query_len, cache, bt, ctx, scale, out
    args = [GOOD, GOOD, 100, 50, cache, GOOD, GOOD, 0.1, GOOD]
    if not torch().cuda.is_available():
        assert prefill(prob, half, args) in (5, 6)
    assert prefill(prob, None, args) == 1
    assert prefill(prob, lib.score(softcap=5.0), args) == 2  # fp32 out
    for i, bad, status in [(0, None, 1), (1, None, 1), (2, -1, 1), (3, -1, 1), (4, None, 1),
                           (5, None, 1), (6, None, 1), (8, None, 1), (7, float("inf"), 1),
                           (0, GOOD + 8, 3), (8, GOOD + 4, 3), (1, GOOD + 2, 3)]:
        a = list(args)
        a[i] = bad
        assert prefill(prob, half, a) == status, (i, bad)
    for i in range(4):
        for bad, status in ((None, 1), (GOOD + 8, 3)):
            parts = [GOOD] * 4
            parts[i] = bad
            a = list(args)
            a[4] = lib.quant_cache(*parts)
            assert prefill(prob, half, a) == status
    for kw, status in [(dict(softcap=-1.0), 1), (dict(window=-1), 1), (dict(prefix_lengths=GOOD + 2), 3),
                       (dict(first_tokens=GOOD + 1), 3)]:
        assert prefill(prob, lib.score(out="fp16", **kw), args) == status, kw
    assert prefill(lib.problem(4, 32, 8, 96, 16, 256, 1024), half, args) == 2
    assert prefill(lib.problem(4, 129, 1, 64, 16, 256, 1024), half, args) == 2
    assert prefill(prob, half, args, opts=lib.options(stages=2)) == 1
    assert prefill(lib.problem(0, 32, 8, 128, 16, 256, 1024), half, args) == 0
    a = list(args)
    a[2] = 0
    assert prefill(prob, half, a) == 0
