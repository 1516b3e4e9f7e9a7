"""pa_prefill_scored (several new tokens per sequence with capped, biased and masked scores)
against the formula in 64 bits, where it can go wrong; refusals on the host; and a layer's run of
append, multi-token attention and decode steps as they are used together."""

import numpy as np
import pytest

from paged_kv_cache_63_gb300 import lib
from tests.gpu_util import torch
from tests.scored_reference import Cached, Rule, assert_within, attend, device_rule, slopes_of

gpu = pytest.mark.gpu
GOOD = 1 << 20

# a probability meets V rounded to fp16 (half a step), relative to a reference that the largest
# is not below: smaller ones are told from 0 down to 2^-25 of it. The capped score is off by the
# polynomial's 6.3e-7 and the roundings of its evaluation; a bias is formed from the tile's
# start (up to 128 tokens away) and the column.
ERRORS = dict(probability_error=2.0 ** -11, weight_floor=2.0 ** -25,
              cap_error=6.3e-7 + 2.0 ** -22, span=128)


def gpu_prefill(w, rule, opts=None, d=None, max_query_len=None, stream=None):
    t = torch()
    d = d or w.to_device()
    o = t.full((w.rows, w.query_heads, w.head_dim), float("nan"), device="cuda", dtype=t.float16)
    most = int(w.new.max()) if max_query_len is None else max_query_len
    lib.pa_prefill_scored(w.prob(), device_rule(rule, "fp16"), d["q"], d["qs"], w.rows, most,
                          d["k"], d["v"], d["bt"], d["ctx"], w.scale, o, opts, stream=stream)
    t.cuda.synchronize()
    return o.cpu().numpy(), lib.pa_get_device_error()


def check(w, rule, **kw):
    got, flags = gpu_prefill(w, rule, **kw)
    assert flags == 0
    want, bound = attend(w, rule, **ERRORS)
    assert np.isnan(got[np.isnan(want)]).all()  # rows of no new token are left alone
    return assert_within(got, want, bound, True)


SHAPES = {
    "hd64_g2": dict(qh=4, kvh=2, hd=64, ps=16),
    "hd128_g4": dict(qh=8, kvh=2, hd=128, ps=16),
    "hd128_g1": dict(qh=2, kvh=2, hd=128, ps=8),
    "hd128_g6": dict(qh=6, kvh=1, hd=128, ps=256),
    "hd256_g6": dict(qh=6, kvh=1, hd=256, ps=64),
    "hd256_g1": dict(qh=2, kvh=2, hd=256, ps=32),
}
CTX = [300, 1, 129, 200, 0, 77]
NEW = [300, 1, 60, 0, 0, 77]


def case(shape, seed=1, **kw):
    args = dict(ctx=CTX, new=NEW, q_scale=3.0, seed=seed, pad=3)
    args.update(SHAPES[shape])
    args.update(kw)
    return Cached(args.pop("ctx"), args.pop("new"), **args)


def documents(w, length):
    """First tokens of documents of about `length`, a row each."""
    rng = np.random.default_rng(5)
    first = np.zeros(w.rows, dtype=np.int32)
    for b in range(w.batch):
        starts = np.concatenate([[0], np.cumsum(rng.integers(1, 2 * length, 400))])
        for row, pos in w.rows_of(b):
            first[row] = starts[starts <= pos].max()
    return first


def rules(w):
    qh = w.query_heads
    return {
        "none": Rule(),
        "cap": Rule(softcap=20.0),
        "cap_low": Rule(softcap=1.5),
        "window1": Rule(window=1),
        "window50": Rule(window=50),
        "window128": Rule(window=128),
        "slopes": Rule(slopes=slopes_of(qh)),
        "documents": Rule(first=documents(w, 30)),
        "prefix": Rule(prefix=np.array([150, 1, 100, 200, 0, 500])),
        "prefix_slopes_cap": Rule(prefix=np.array([150, 0, 129, -4, 3, 40]), slopes=slopes_of(qh),
                                  softcap=5.0),
        "all": Rule(softcap=3.0, window=90, slopes=slopes_of(qh), first=documents(w, 100),
                    prefix=np.array([130, 1, 80, 0, 0, 70])),
    }


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
    """Cap, slopes and first tokens have kernels for each combination of them; windows and prefixes
    go through all."""
    w = case(shape, ctx=[150, 70, 3], new=[150, 20, 3], seed=parts)
    rule = dict(softcap=4.0 if parts & 1 else 0.0,
                slopes=slopes_of(w.query_heads) if parts & 2 else None,
                first=documents(w, 25) if parts & 4 else None)
    check(w, Rule(**rule))
    check(w, Rule(window=40, prefix=np.array([90, 0, 2]), **rule))


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g1", "hd256_g1"])
def test_one_new_token_each(shape):
    w = case(shape, ctx=[1, 2, 128, 129, 400, 257], new=[1] * 6)
    for rule in (Rule(softcap=5.0), Rule(window=130), Rule(first=np.array([0, 1, 127, 128, 3, 250, 0, 0, 0]))):
        check(w, rule)


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd128_g1", "hd256_g6"])
def test_rows_that_see_nothing_are_zero(shape):
    """Single rows, whole query tiles, and a row between rows that see much."""
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
    """Chunks on long prefixes: pages before every row's window have left the table, and slots
    that stay hold NaN and Inf."""
    w = case(shape, ctx=[700, 411, 129], new=[90, 1, 129], pad=0)
    rule = Rule(window=window, softcap=10.0)
    want = attend(w, rule, **ERRORS)
    for b in range(w.batch):
        w.forget(b, max(0, int(w.ctx[b] - w.new[b]) - window + 1))
    got, flags = gpu_prefill(w, rule)
    assert flags == 0
    assert_within(got, *want, True)


@gpu
@pytest.mark.parametrize("shape", ["hd128_g4", "hd256_g6"])
def test_non_finite_keys_of_unseen_documents(shape):
    """A finished document's keys and values may be anything once no new token sees them."""
    w = case(shape, ctx=[500, 300], new=[100, 44], pad=0)
    first = np.concatenate([np.full(100, 387), np.full(44, 255)])
    rule = Rule(first=first, slopes=slopes_of(w.query_heads))
    want = attend(w, rule, **ERRORS)
    w.forget(0, 387)
    w.forget(1, 255)
    got, flags = gpu_prefill(w, rule)
    assert flags == 0
    assert_within(got, *want, True)


@gpu
@pytest.mark.parametrize("prefix", [0, 560])
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd128_g6", "hd256_g6", "hd256_g1"])
def test_tokens_nobody_sees_between_seen_ones(shape, prefix):
    """Rows that see nothing leave their own tokens unseen, between tokens that other rows of the
    same work item see: their slots hold NaN and Inf, and pages of nothing else have left the
    table."""
    w = case(shape, ctx=[700, 411, 130], new=[200, 150, 130], pad=0)
    first = np.zeros(w.rows, dtype=np.int64)
    never = 1 << 30
    first[5:40] = never                       # the first sequence: the old tokens, then two holes
    first[40:150] = 540 + np.arange(110) // 2
    first[150:195] = never
    first[195:200] = 699                      # and rows that see the last token or nothing
    at = 200
    for j in range(150):                      # the second: every third row sees itself alone
        first[at + j] = 411 - 150 + j if j % 3 == 0 else never
    first[350:420] = never                    # the third: nothing, then from a later token on
    first[420:] = 75
    rule = Rule(first=first, softcap=10.0, prefix=np.array([prefix, 0, 0]))
    want = attend(w, rule, **ERRORS)
    for b in range(w.batch):
        n = int(w.ctx[b])
        seen = np.zeros(n + w.ps, dtype=bool)
        for row, pos in w.rows_of(b):
            seen[first[row]:max(pos + 1, int(rule.prefix[b]) if pos < rule.prefix[b] else 0)] = True
        for t in range(n):
            if not seen[t]:
                w.k[w.bt[b, t // w.ps], t % w.ps] = np.nan
                w.v[w.bt[b, t // w.ps], t % w.ps] = np.inf
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
    values, which would take another form of tanh."""
    w = case(shape, ctx=[300, 1, 129, 200], new=[170, 1, 60, 31], q_scale=1.0, pad=5)
    rule = Rule(softcap=20.0, window=100, slopes=slopes_of(w.query_heads) if slopes else None)
    for b in range(w.batch):
        w.forget(b, max(0, int(w.ctx[b] - w.new[b]) - rule.window + 1))
    rows, unseen = int(w.qs[-1]), np.isnan(w.k)
    outs = []
    for fill in (0.0, 3000.0, np.nan):
        w.k[unseen] = fill
        w.q[rows:] = fill
        out, flags = gpu_prefill(w, rule)
        assert flags == 0
        outs.append(out[:rows].view(np.uint16))
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_growing_maxima_and_scores_past_the_polynomial(shape):
    w = case(shape, ctx=[600, 300], new=[500, 300], pad=0)
    for b in range(w.batch):
        for t in range(int(w.ctx[b])):
            page, slot = w.bt[b, t // w.ps], t % w.ps
            w.k[page, slot] = (w.k[page, slot].astype(np.float32) * (1 + t / 60)).astype(np.float16)
    check(w, Rule())
    check(w, Rule(softcap=20.0))
    check(w, Rule(softcap=500.0, window=250))
    check(w, Rule(slopes=-0.05 * slopes_of(w.query_heads), first=documents(w, 150)))


@gpu
def test_negative_scale_and_steep_biases():
    w = case("hd128_g4")
    w.scale = -w.scale
    check(w, Rule())
    check(w, Rule(window=140))
    check(w, Rule(softcap=6.0, slopes=100.0 * slopes_of(w.query_heads)))
    w.scale = 0.0  # every seen token weighs the same
    check(w, Rule(window=70))
    check(w, Rule(softcap=6.0))
    check(w, Rule(slopes=slopes_of(w.query_heads)))


@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_grid_taller_than_needed_and_unaligned_output(shape):
    t = torch()
    w = case(shape)
    check(w, Rule(softcap=9.0, prefix=w.ctx), max_query_len=900)
    d, rule = w.to_device(), Rule(window=100)
    n = w.rows * w.query_heads * w.head_dim
    flat = t.zeros(n + 8, device="cuda", dtype=t.float16)  # 16-byte but not 32-byte aligned
    o = flat[8:].view(w.rows, w.query_heads, w.head_dim)
    assert o.data_ptr() % 32 == 16
    lib.pa_prefill_scored(w.prob(), device_rule(rule, "fp16"), d["q"], d["qs"], w.rows, 300, d["k"],
                          d["v"], d["bt"], d["ctx"], w.scale, o)
    t.cuda.synchronize()
    assert lib.pa_get_device_error() == 0
    assert_within(o.cpu().numpy(), *attend(w, rule, **ERRORS), True)


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
    call = lambda: lib.pa_prefill_scored(  # noqa: E731
        w.prob(), dr, d["q"], d["qs"], w.rows, int(w.new.max()), d["k"], d["v"], d["bt"], d["ctx"],
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
    """Work items of one to four key tiles, hundreds to an SM, in an order that gives every warp
    items without a tile of its own between others: repeated calls give the same rows."""
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
            lib.pa_prefill_scored(w.prob(), dr, d["q"], d["qs"], w.rows, 300, d["k"], d["v"], d["bt"],
                                  d["ctx"], w.scale, o, stream=s)
    t.cuda.synchronize()
    live = ~np.isnan(want[0])
    for o in outs:
        assert_within(o.cpu().numpy(), want[0], want[1], True)
        assert (o.cpu().numpy()[~live] == 0).all()


@gpu
@pytest.mark.parametrize("shape", ["hd128_g4", "hd256_g6"])
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
@pytest.mark.parametrize("shape", ["hd128_g4", "hd256_g6"])
def test_expired_wait_is_reported(shape):
    w = case(shape)
    _, flags = gpu_prefill(w, Rule(softcap=5.0), lib.options(test_flags=lib.PA_TEST_EXPIRE_WAITS))
    assert flags & lib.PA_DEVERR_TIMEOUT
    check(w, Rule(softcap=5.0))


# ---------------------------------------------------------------------------- a layer's run
@gpu
@pytest.mark.parametrize("shape", ["hd64_g2", "hd128_g4", "hd256_g6"])
def test_append_prefill_and_decode_steps_together(shape):
    """As a serving loop runs a local layer: prompts appended (keys turned by position) and
    attended, then decode steps, each an append of one token and a scored decode. Every output is
    checked against the formula over the cache the calls themselves wrote, and the cache against
    the rotation by the host."""
    from tests.test_append_rope import Case

    t = torch()
    steps, lens = 4, np.array([130, 5, 64])
    s = SHAPES[shape]
    final = Cached(lens + steps, np.zeros(3, dtype=int), **s)  # pages for the whole run
    d = final.to_device()
    table = Case([1], [int(lens.max()) + steps], hd=s["hd"]).table
    rope = lib.rope(s["hd"], "half", t.from_numpy(table).cuda())
    rng = np.random.default_rng(3)
    rule = Rule(softcap=12.0, window=60)
    prob = final.prob()
    n_ws = lib.pa_workspace_size(prob)
    ws = t.empty(max(n_ws, 256), dtype=t.uint8, device="cuda")
    qh, kvh, hd = s["qh"], s["kvh"], s["hd"]
    for step in range(steps + 1):
        new = lens if step == 0 else np.ones(3, dtype=int)
        ctx = lens + step
        rows = int(new.sum())
        qkv = t.from_numpy(rng.standard_normal((rows, qh + 2 * kvh, hd)).astype(np.float16)).cuda()
        qs = t.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
        dctx = t.from_numpy(ctx.astype(np.int32)).cuda()
        q = t.empty(rows, qh, hd, dtype=t.float16, device="cuda")
        o = t.empty_like(q)
        lib.pa_append_rope(prob, rope, qkv[:, :qh], qkv[:, qh:qh + kvh], qkv[:, qh + kvh:], qs, rows,
                           d["bt"], dctx, q, d["k"], d["v"])
        dr = device_rule(rule, "fp16")
        if step == 0:
            lib.pa_prefill_scored(prob, dr, q, qs, rows, int(new.max()), d["k"], d["v"], d["bt"],
                                  dctx, final.scale, o)
        else:
            lib.pa_decode_scored(prob, dr, q, d["k"], d["v"], d["bt"], dctx, final.scale, o,
                                 workspace=ws, workspace_bytes=n_ws)
        t.cuda.synchronize()
        assert lib.pa_get_device_error() == 0
        now = final
        now.ctx, now.new, now.rows = ctx.astype(np.int32), new, rows
        now.qs = qs.cpu().numpy()
        now.q, now.k, now.v = (x.cpu().numpy() for x in (q, d["k"], d["v"]))
        # the newest keys are the projection's, turned (bounds as in test_append_rope)
        host = Case(new, ctx, qh=qh, kvh=kvh, hd=hd)
        host.qkv, host.table = qkv.cpu().numpy(), table
        for b in range(3):
            row, pos = now.rows_of(b)[-1]
            x, slack = host.turned([row], [pos])
            at = (now.bt[b, pos // now.ps], pos % now.ps)
            assert (np.abs(now.k[at].astype(np.float64) - x[0, qh:]) <= slack[0, qh:]).all()
            assert np.array_equal(now.v[at], host.qkv[row, qh + kvh:])
        assert_within(o.cpu().numpy(), *attend(now, rule, **ERRORS), True)


@gpu
@pytest.mark.parametrize("head_major", [0, 1])
def test_pages_past_32_bit_offsets(head_major):
    """Appended to, and attended from, pages that lie more than 2^31 elements into the caches: the
    same bits as from a small cache."""
    t = torch()
    qh, kvh, hd, ps = 16, 8, 256, 256
    ctx, rows = [400, 300], 700
    far = 4300  # pages of 2^19 elements
    scale, rope_dim = 0.0625, 64
    g = t.Generator(device="cuda").manual_seed(5)
    qkv = t.randn(rows, qh + 2 * kvh, hd, generator=g, device="cuda", dtype=t.float16)
    ang = t.rand(512, rope_dim // 2, generator=g, device="cuda") * 6
    rope = lib.rope(rope_dim, "interleaved", t.stack([ang.cos(), ang.sin()], 1).contiguous())
    put = lambda x: t.tensor(x, dtype=t.int32, device="cuda")  # noqa: E731
    qs, dctx = put([0, 400, 700]), put(ctx)
    shape = (kvh, ps, hd) if head_major else (ps, kvh, hd)
    outs = []
    for pages, table in [(4, [[2, 0], [3, 1]]), (far, [[far - 1, 4097], [4, far - 2]])]:
        k, v = (t.empty((pages, *shape), dtype=t.float16, device="cuda") for _ in range(2))
        bt = put(table)
        prob = lib.problem(2, qh, kvh, hd, ps, 2, pages, head_major)
        q = t.empty(rows, qh, hd, dtype=t.float16, device="cuda")
        o, last = t.empty_like(q), t.empty(2, qh, hd, dtype=t.float16, device="cuda")
        rule = lib.score(softcap=20.0, window=150, out="fp16")
        lib.pa_append_rope(prob, rope, qkv[:, :qh], qkv[:, qh:qh + kvh], qkv[:, qh + kvh:], qs, rows,
                           bt, dctx, q, k, v)
        lib.pa_prefill_scored(prob, rule, q, qs, rows, 400, k, v, bt, dctx, scale, o)
        n = lib.pa_workspace_size(prob)
        ws = t.empty(max(n, 256), dtype=t.uint8, device="cuda")
        lib.pa_decode_scored(prob, rule, q[[399, 699]].contiguous(), k, v, bt, dctx, scale, last,
                             workspace=ws, workspace_bytes=n)
        t.cuda.synchronize()
        assert lib.pa_get_device_error() == 0
        outs.append([x.cpu().numpy() for x in (q, o, last, k[bt[:, 0].long()])])
        del k, v
        t.cuda.empty_cache()
    for small, large in zip(*outs):
        assert np.isfinite(small).all()
        assert np.array_equal(small.view(np.uint16), large.view(np.uint16))
    # the newest token of each sequence, both ways: two outputs below 8 rounded to fp16 (2^-9 each)
    # and weights rounded to fp16 (2^-11 of values below 8)
    a, b = outs[1][1][[399, 699]], outs[1][2]
    assert np.abs(a).max() < 8 and np.abs(a.astype(np.float64) - b).max() < 2 * 2 ** -9 + 2 ** -8


# ---------------------------------------------------------------------------- refusals
def prefill(prob, score, a, **kw):
    return lib.status_of(lib.pa_prefill_scored, prob, score, *a, **kw)


def test_refusals():
    prob = lib.problem(4, 32, 8, 128, 16, 256, 1024)
    half = lib.score(softcap=5.0, out="fp16")
    # query, query_start, total_tokens, max_query_len, k, v, bt, ctx, scale, out
    args = [GOOD, GOOD, 100, 50, GOOD, GOOD, GOOD, GOOD, 0.1, GOOD]
    if not torch().cuda.is_available():
        assert prefill(prob, half, args) in (5, 6)
    assert prefill(prob, None, args) == 1
    assert prefill(prob, lib.score(softcap=5.0), args) == 2  # fp32 out
    for i, bad, status in [(0, None, 1), (1, None, 1), (2, -1, 1), (3, -1, 1), (4, None, 1),
                           (9, None, 1), (8, float("inf"), 1), (0, GOOD + 8, 3), (9, GOOD + 4, 3),
                           (1, GOOD + 2, 3)]:
        a = list(args)
        a[i] = bad
        assert prefill(prob, half, a) == status, (i, bad)
    for kw, status in [(dict(softcap=-1.0), 1), (dict(softcap=float("nan")), 1), (dict(window=-1), 1),
                       (dict(prefix_lengths=GOOD + 2), 3), (dict(first_tokens=GOOD + 1), 3)]:
        assert prefill(prob, lib.score(out="fp16", **kw), args) == status, kw
    assert prefill(lib.problem(4, 32, 8, 96, 16, 256, 1024), half, args) == 2
    assert prefill(lib.problem(4, 129, 1, 64, 16, 256, 1024), half, args) == 2
    assert prefill(prob, half, args, opts=lib.options(stages=2)) == 1
    assert prefill(lib.problem(0, 32, 8, 128, 16, 256, 1024), half, args) == 0
    a = list(args)
    a[2] = 0
    assert prefill(prob, half, a) == 0


def test_no_rows_need_no_addresses():
    """An empty tensor's address is null."""
    prob = lib.problem(4, 32, 8, 128, 16, 256, 1024)
    half = lib.score(softcap=5.0, out="fp16")
    args = [None, GOOD, 0, 0, GOOD, GOOD, GOOD, GOOD, 0.1, None]
    assert prefill(prob, half, args) == 0
    args[2] = args[3] = 1
    assert prefill(prob, half, args) == 1
    assert prefill(prob, half, [None, GOOD, 0, 0, None, GOOD, GOOD, GOOD, 0.1, None]) == 1
    assert prefill(prob, half, [None, GOOD, 0, 0, GOOD, None, GOOD, GOOD, 0.1, None]) == 1
