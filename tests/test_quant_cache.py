"""pa_append_quant and pa_read_quant against the format in 64 bits: codes and scales exactly, queries
within the roundings of fp32 and fp16; refusals on the host."""

import numpy as np
import pytest

from paged_kv_cache_63_gb300 import lib
from tests.gpu_util import torch
from tests.quant_reference import GRID, numbers, quantise, scale_layout
from tests.test_append_rope import CASES, GOOD, Case

gpu = pytest.mark.gpu
EPS = 1e-6


class QuantCase(Case):
    """One call's inputs on the host; every code, scale and output row starts out random."""

    def __init__(self, new, ctx, norm="both", seed=0, **kw):
        super().__init__(new, ctx, seed=seed, **kw)
        rng = np.random.default_rng(seed + 5)
        self.codes, self.scales = {}, {}
        for x in "kv":
            c = rng.integers(0, 256, (self.pages, self.ps, self.kvh, self.hd)).astype(np.uint8)
            c[(c & 127) == 127] = 5
            self.scales[x] = rng.integers(112, 136, c.shape[:-1]).astype(np.uint8)
            # the format has no code above 240 under 2^8 (no number of fp16 needs one)
            self.codes[x] = np.where((self.scales[x] == 135)[..., None] & ((c & 127) > 0x77), 3, c)
        w = lambda: (1.0 + 0.3 * rng.standard_normal(self.hd)).astype(np.float32)  # noqa: E731
        self.q_weight = w() if norm in ("both", "query") else None
        self.k_weight = w() if norm in ("both", "key") else None

    def device_codes(self, x):
        return np.ascontiguousarray(x.transpose(0, 2, 1, 3)) if self.head_major else x

    def exact(self, row, pos):
        """The row's query and key heads normed and turned in 64 bits, and a bound of the pairs'
        size that fp32 errors are relative to."""
        x = self.qkv[row, :self.qh + self.kvh].astype(np.float64)
        for heads, w in ((slice(0, self.qh), self.q_weight), (slice(self.qh, None), self.k_weight)):
            if w is not None:
                size = np.sqrt((x[heads] ** 2).mean(-1, keepdims=True) + np.float64(np.float32(EPS)))
                x[heads] = x[heads] / size * w.astype(np.float64)
        out, both = x.copy(), np.abs(x)
        r = self.rotary
        if r:
            i = np.arange(0, r, 2) if self.interleaved else np.arange(r // 2)
            j = i + (1 if self.interleaved else r // 2)
            c, s = (self.table[pos, k].astype(np.float64) for k in (0, 1))
            out[..., i] = x[..., i] * c - x[..., j] * s
            out[..., j] = x[..., i] * s + x[..., j] * c
            both[..., i] = both[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
        return out, both

    def expected(self, skip=()):
        """(queries, their bound, codes and scales of keys and values as numbers)."""
        q, tol = self.q_out.astype(np.float64), np.zeros(self.q_out.shape)
        codes = {x: c.copy() for x, c in self.codes.items()}
        scales = {x: c.copy() for x, c in self.scales.items()}
        for b, n in enumerate(self.new):
            for j in range(int(n)):
                row, t = int(self.qs[b]) + j, int(self.ctx[b] - n + j)
                if row in skip:
                    continue
                pos = int(self.positions[row]) if self.positions is not None else t
                x, both = self.exact(row, pos)
                q[row] = x[:self.qh]
                # at most 16 roundings of fp32 of the pair, then half a step of fp16
                tol[row] = (both[:self.qh] * 2.0 ** -20
                            + (np.abs(x[:self.qh]) + both[:self.qh] * 2.0 ** -20) * 2.0 ** -11
                            + 2.0 ** -25)
                at = (int(self.bt[b, t // self.ps]), t % self.ps)
                codes["k"][at], scales["k"][at] = quantise(x[self.qh:])
                codes["v"][at], scales["v"][at] = quantise(self.qkv[row, self.qh + self.kvh:])
        return q, tol, codes, scales

    def put(self, **changed):
        t = torch()
        h = {n: getattr(self, n) for n in ("qkv", "qs", "bt", "ctx", "q_out", "table", "positions",
                                           "q_weight", "k_weight")}
        for x in "kv":
            h[x] = self.device_codes(self.codes[x])
            h[x + "s"] = scale_layout(self.scales[x])
        h.update(changed)
        return {n: None if a is None else t.from_numpy(np.ascontiguousarray(a)).cuda()
                for n, a in h.items()}

    def call(self, d, with_query=True, in_place=False, stream=None):
        qh, kvh = self.qh, self.kvh
        parts = [d["qkv"][:, :qh], d["qkv"][:, qh:qh + kvh], d["qkv"][:, qh + kvh:]]
        if not self.fused:
            parts = [p.contiguous() for p in parts]
        if in_place:
            d["q_out"] = parts[0]
        rope = lib.rope(self.rotary, "interleaved" if self.interleaved else "half", d["table"],
                        d["positions"])
        norm = None
        if d["q_weight"] is not None or d["k_weight"] is not None:
            norm = lib.norm(EPS, d["q_weight"], d["k_weight"])
        lib.pa_append_quant(self.prob(), norm, rope, parts[0] if with_query else None, parts[1],
                            parts[2], d["qs"], self.total, d["bt"], d["ctx"],
                            d["q_out"] if with_query else None,
                            lib.quant_cache(d["k"], d["v"], d["ks"], d["vs"]), stream=stream)

    def results(self, d):
        """(queries, codes, scales) as [page][slot][kv_head]..., and the flags."""
        torch().cuda.synchronize()
        back = lambda a: a.transpose(0, 2, 1, 3) if self.head_major else a  # noqa: E731
        codes = {x: back(d[x].cpu().numpy()) for x in "kv"}
        scales = {x: d[x + "s"].cpu().numpy().transpose(0, 2, 1) for x in "kv"}
        return (d["q_out"].cpu().numpy(), codes, scales), lib.pa_get_device_error()

    def run(self, with_query=True, in_place=False, stream=None, **changed):
        d = self.put(**changed)
        self.call(d, with_query, in_place, stream)
        return self.results(d)


def check(case, got, flags=0, want_flags=0, skip=(), queries=True):
    assert flags == want_flags
    q, tol, codes, scales = case.expected(skip)
    if queries:
        err = np.abs(got[0].astype(np.float64) - q)
        assert (err <= tol).all(), f"query: {int((err > tol).sum())} of {err.size}, {err.max()}"
    for x in "kv":
        assert np.array_equal(got[2][x], scales[x]), f"scales of {x}"
        a, b = numbers(got[1][x], scales[x]), numbers(codes[x], scales[x])
        assert np.array_equal(a, b), f"{x}: {int((a != b).sum())} of {a.size} codes"


# ---------------------------------------------------------------------------- the format
def test_the_reference_holds_what_it_says():
    """Values of fp16, of every size, come back within half a step; the largest elements and ties."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)) * 2.0 ** rng.integers(-24, 16, (200, 1))
    x = x.clip(-65504, 65504).astype(np.float16).astype(np.float64)
    c, s = quantise(x)
    y = numbers(c, s)
    step = np.maximum(np.abs(x) * np.where(np.abs(x) > 61440, 2.0 ** -3.9, 2.0 ** -4), 2.0 ** -10 * 2.0 ** (s.astype(float) - 127)[:, None])
    assert (np.abs(y - x) <= step).all()
    assert np.array_equal(y.astype(np.float16).astype(np.float64), y)  # fp16 numbers
    assert (np.abs(y) <= 61440).all()
    for top, e, want in [(0, -15, 0), (448 * 2.0 ** -15, -15, 448 * 2.0 ** -15),
                         (449 * 2.0 ** -15, -14, 448 * 2.0 ** -15), (1.75, -8, 1.75),
                         (1.8, -7, 1.75), (448, 0, 448), (57344, 7, 57344), (57376, 8, 57344),
                         (65504, 8, 61440)]:
        row = np.zeros(64)
        row[5] = -top
        c, s = quantise(row)
        assert s == e + 127 and numbers(c, s)[5] == -want
    tie = np.array([448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])  # even codes: 16, 20, 0, 2^-8
    c, s = quantise(tie)
    assert numbers(c, s).tolist() == [448.0, 16.0, 20.0, 0.0, 2.0 ** -8]
    assert GRID[126] == 448


# ---------------------------------------------------------------------------- append
@gpu
@pytest.mark.parametrize("head_major", [0, 1])
@pytest.mark.parametrize("norm", ["both", "none"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_matches_the_format(name, norm, head_major):
    case = QuantCase(norm=norm, head_major=head_major, **CASES[name])
    check(case, *case.run())


@gpu
@pytest.mark.parametrize("norm", ["query", "key"])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_one_kind_of_rows_normed(norm, hd):
    case = QuantCase([7, 2], [33, 2], norm=norm, hd=hd, rotary=32, qh=6, kvh=3)
    check(case, *case.run())


@gpu
@pytest.mark.parametrize("head_major,hd,qh,kvh,ps,interleaved", [
    (0, 64, 2, 1, 8, False), (1, 64, 14, 2, 16, True), (0, 128, 3, 3, 16, False),
    (1, 256, 2, 1, 64, False), (0, 256, 1, 1, 32, True)])
def test_many_rows(head_major, hd, qh, kvh, ps, interleaved):
    """Many rows, ragged, rows of a padded batch among the last."""
    rng = np.random.default_rng(3)
    ctx = rng.integers(1, 300, 56)
    new = np.minimum(ctx, rng.integers(0, 300, 56))
    new[3] = ctx[3] = 2000
    new[40] = ctx[40] = 8192 - 2 - new.sum() + new[40] + 5
    case = QuantCase(new, ctx, qh=qh, kvh=kvh, hd=hd, ps=ps, head_major=head_major,
                     interleaved=interleaved, pad=3, explicit=bool(head_major))
    assert case.total >= 8192
    check(case, *case.run())
    bt = case.bt.copy()  # a page outside the pool, in the middle
    bt[3, 5] = -7
    hit = {int(case.qs[3]) + j for j in range(2000) if j // ps == 5}
    check(case, *case.run(bt=bt), want_flags=lib.PA_DEVERR_PAGE_ID, skip=hit)
    case.fused, case.q_out = False, np.ascontiguousarray(case.qkv[:, :qh])
    check(case, *case.run(in_place=True))
    got, flags = case.run(with_query=False)
    check(case, got, flags, queries=False)


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_keys_on_the_border_of_two_codes(interleaved):
    """Unturned and unnormed keys that lie between two codes, or next to there by the smallest
    step of fp16; and turned by a quarter of a circle, which moves them to other elements exactly."""
    rng = np.random.default_rng(1)
    mid = (GRID[8:126] + GRID[9:127]) / 2
    rows = np.zeros((40, 1, 64))
    for r in rows:
        x = rng.choice(mid, 64) * rng.choice([-1, 1], 64)
        bits = (x.astype(np.float16).view(np.int16) + rng.integers(-1, 2, 64)).astype(np.int16)
        r[0] = bits.view(np.float16)
        r[0, 7] = 448.0
    case = QuantCase([40], [40], qh=1, kvh=1, norm="none", interleaved=interleaved)
    case.qkv[:, 1:2] = rows
    case.qkv[:, 2:3] = -rows
    case.table[:, 0], case.table[:, 1] = 0.0, 1.0
    check(case, *case.run())
    case.rotary, case.table = 0, case.table[:, :, :0]
    check(case, *case.run())


@gpu
def test_rows_of_every_size():
    """Rows of zeroes, of fp16's largest and smallest numbers, and largest elements on either side of
    where the scale steps."""
    case = QuantCase([64], [64], qh=2, kvh=2, norm="none", rotary=0)
    rng = np.random.default_rng(2)
    for r in range(64):
        for h in (2, 3, 4, 5):
            x = rng.standard_normal(64) * 2.0 ** rng.integers(-26, 14)
            kind = (r + h) % 8
            if kind == 0:
                x[:] = 0.0
            elif kind == 1:
                x[rng.integers(64)] = rng.choice([65504.0, -65504.0, 61440.0, 63488.0, 57344.0])
            elif kind == 2:
                x[:] = rng.integers(-3, 4, 64) * 2.0 ** -24
            elif kind == 3:
                top = np.float16(448 * 2.0 ** rng.integers(-15, 8))
                x = np.clip(x, -top / 2, top / 2)
                x[5] = -np.uint16(int(top.view(np.uint16)) + rng.integers(-1, 2)).view(np.float16)
            elif kind == 4:
                x[::2] = -0.0
            case.qkv[r, h] = np.clip(x, -65504, 65504).astype(np.float16)
    check(case, *case.run())


@gpu
def test_a_row_that_is_not_finite_leaves_the_others_alone():
    case = QuantCase([9, 3], [9, 3], qh=4, kvh=4, hd=128)
    for value in (np.nan, np.inf, -np.inf):
        qkv = case.qkv.copy()
        qkv[4, 4 + 1, 17] = value       # a key
        qkv[2, 8 + 1, 100] = value      # a value
        got, flags = case.run(qkv=qkv)
        q, tol, codes, scales = case.expected()
        assert flags == 0 and (np.abs(got[0] - q) <= tol).all()
        for x, row, head in (("k", 4, 1), ("v", 2, 1)):
            at = (int(case.bt[0, row // case.ps]), row % case.ps, head)
            a, b = numbers(got[1][x], got[2][x]), numbers(codes[x], scales[x])
            a[at] = b[at] = 0
            got[2][x][at] = scales[x][at]
            assert np.array_equal(a, b) and np.array_equal(got[2][x], scales[x])


@gpu
@pytest.mark.parametrize("pad", [0, 2])
def test_no_new_tokens(pad):
    for fused in (True, False):
        case = QuantCase([0, 0], [40, 3], pad=pad, fused=fused)
        check(case, *case.run())


@gpu
def test_keys_and_values_alone_and_queries_in_place():
    case = QuantCase([5, 3], [40, 3])
    got, flags = case.run(with_query=False)
    assert np.array_equal(got[0], case.q_out)
    check(case, got, flags, queries=False)
    case = QuantCase([5, 3, 0, 9], [40, 3, 0, 9], fused=False, pad=2)
    got, flags = case.run(in_place=True)
    case.q_out = np.ascontiguousarray(case.qkv[:, :case.qh])  # rows behind the last stay
    check(case, got, flags)


@gpu
def test_bad_sequences_and_tokens_are_flagged_and_skipped():
    case = QuantCase([4, 4, 4, 4, 4], [20, 30, 40, 12, 8], pad=1)
    ctx_out = case.ctx.copy()
    ctx_out[1], ctx_out[3] = -1, case.maxp * case.ps + 1
    qs_past = case.qs.copy()
    qs_past[-1] = case.total + 1
    for changed, flag, bad in [(dict(ctx=ctx_out), lib.PA_DEVERR_CONTEXT, (1, 3)),
                               (dict(qs=qs_past), lib.PA_DEVERR_QUERY_START, (4,))]:
        rows = {r for b in bad for r in range(4 * b, 4 * b + 4)}
        check(case, *case.run(**changed), want_flags=flag, skip=rows)
    bt = case.bt.copy()
    bt[1, 29 // case.ps] = case.pages
    hit = {4 + j for j in range(4) if (26 + j) // case.ps == 29 // case.ps}
    check(case, *case.run(bt=bt), want_flags=lib.PA_DEVERR_PAGE_ID, skip=hit)
    pos = np.zeros(case.total, dtype=np.int32)
    pos[2], pos[7] = -1, case.table.shape[0]
    case.positions = pos
    check(case, *case.run(), want_flags=lib.PA_DEVERR_POSITION, skip={2, 7})


@gpu
@pytest.mark.parametrize("rows", [64, 8300])
def test_captured_and_replayed_with_new_inputs_on_another_stream(rows):
    t = torch()
    case = QuantCase([rows, 3], [rows, 64], qh=2, kvh=1)
    d = case.put()
    case.call(d)
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        case.call(d)
    for seed in (3, 4):
        case.qkv = np.random.default_rng(seed).standard_normal(case.qkv.shape).astype(np.float16)
        d["qkv"].copy_(t.from_numpy(case.qkv))
        t.cuda.synchronize()
        s = t.cuda.Stream()
        with t.cuda.stream(s):
            g.replay()
        check(case, *case.results(d))


# ---------------------------------------------------------------------------- read
def read(case, d, k=True, v=True, fill=7.0):
    t = torch()
    out = [t.full((case.total, case.kvh, case.hd), fill, dtype=t.float16, device="cuda")
           if want else None for want in (k, v)]
    lib.pa_read_quant(case.prob(), lib.quant_cache(d["k"], d["v"], d["ks"], d["vs"]), d["qs"],
                      case.total, d["bt"], d["ctx"], *out)
    t.cuda.synchronize()
    return [None if o is None else o.cpu().numpy() for o in out], lib.pa_get_device_error()


def rows_read(case, x, skip=(), fill=7.0):
    out = np.full((case.total, case.kvh, case.hd), fill)
    for b, n in enumerate(case.new):
        for j in range(int(n)):
            row, t = int(case.qs[b]) + j, int(case.ctx[b] - n + j)
            if row not in skip:
                at = (int(case.bt[b, t // case.ps]), t % case.ps)
                out[row] = numbers(case.codes[x][at], case.scales[x][at])
    return out


@gpu
@pytest.mark.parametrize("head_major", [0, 1])
@pytest.mark.parametrize("name", sorted(CASES))
def test_read_back_exactly(name, head_major):
    case = QuantCase(head_major=head_major, **CASES[name])
    got, flags = read(case, case.put())
    assert flags == 0
    for x, a in zip("kv", got):
        assert np.array_equal(a.astype(np.float64), rows_read(case, x))


@gpu
def test_read_keys_or_values_alone_and_bad_pages():
    case = QuantCase([40, 3, 9], [50, 90, 9], kvh=3, qh=3, pad=2)
    d = case.put()
    for k, v in ((True, False), (False, True)):
        got, flags = read(case, d, k, v)
        assert flags == 0 and (got[0] is None) != k and (got[1] is None) != v
        x = "k" if k else "v"
        assert np.array_equal(got[0 if k else 1].astype(np.float64), rows_read(case, x))
    bt = case.bt.copy()
    bt[0, 1] = 1 << 20
    hit = {j for j in range(40) if (10 + j) // case.ps == 1}
    got, flags = read(case, case.put(bt=bt))
    assert flags == lib.PA_DEVERR_PAGE_ID
    for x, a in zip("kv", got):
        assert np.array_equal(a.astype(np.float64), rows_read(case, x, hit))
    ctx = case.ctx.copy()
    ctx[2] = 5
    got, flags = read(case, case.put(ctx=ctx))
    assert flags == lib.PA_DEVERR_QUERY_START
    for x, a in zip("kv", got):
        assert np.array_equal(a.astype(np.float64), rows_read(case, x, set(range(43, 52))))


@gpu
def test_written_and_read_back():
    """What was appended reads back as the format says, and reading changes nothing."""
    case = QuantCase([30, 0, 5], [30, 9, 77], hd=128, qh=4, kvh=2, ps=32)
    d = case.put()
    case.call(d)
    before = [d[n].clone() for n in ("k", "v", "ks", "vs")]
    got, flags = read(case, d)
    assert flags == 0
    _, _, case.codes, case.scales = case.expected()
    for x, a in zip("kv", got):
        assert np.array_equal(a.astype(np.float64), rows_read(case, x))
    assert all((d[n] == b).all() for n, b in zip(("k", "v", "ks", "vs"), before))


# ---------------------------------------------------------------------------- refusals
def append(prob, norm, rope, cache, **kw):
    a = dict(query=GOOD, new_key=GOOD, new_value=GOOD, query_start=GOOD, total_tokens=10,
             block_tables=GOOD, context_lengths=GOOD, query_out=GOOD + 4096)
    a.update(kw)
    return lib.status_of(lib.pa_append_quant, prob, norm, rope, cache=cache, **a)


def test_refusals():
    prob = lib.problem(4, 8, 2, 64, 16, 8, 32)
    cache = lib.quant_cache(GOOD, GOOD, GOOD, GOOD)
    if not torch().cuda.is_available():
        assert append(prob, None, None, cache) in (5, 6)
        assert append(prob, lib.norm(1e-6, GOOD, GOOD), None, cache) in (5, 6)
    assert append(prob, None, None, None) == 1
    for i in range(4):
        for bad, status in ((None, 1), (GOOD + 8, 3)):
            a = [GOOD] * 4
            a[i] = bad
            assert append(prob, None, None, lib.quant_cache(*a)) == status
            assert lib.status_of(lib.pa_read_quant, prob, lib.quant_cache(*a), GOOD, 10, GOOD, GOOD,
                                 GOOD, GOOD) == status
    for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-31, 1e31):
        assert append(prob, lib.norm(eps, GOOD), None, cache) == 1
    n = lib.norm(1e-6, GOOD)
    n.reserved = 1
    assert append(prob, n, None, cache) == 1
    assert append(prob, lib.norm(1e-6, GOOD + 4), None, cache) == 3
    assert append(prob, lib.norm(1e-6, None, GOOD + 8), None, cache) == 3
    for kw, status in [(dict(new_key=None), 1), (dict(new_value=None), 1), (dict(query=None), 1),
                       (dict(query_out=None), 1), (dict(query_start=None), 1),
                       (dict(block_tables=None), 1), (dict(context_lengths=None), 1),
                       (dict(total_tokens=-1), 1), (dict(total_tokens=1 << 31), 1),
                       (dict(key_stride=64), 1), (dict(value_stride=132), 3),
                       (dict(new_key=GOOD + 8), 3), (dict(context_lengths=GOOD + 2), 3)]:
        assert append(prob, None, None, cache, **kw) == status, kw
    assert append(lib.problem(4, 8, 2, 96, 16, 8, 32), None, None, cache) == 2
    assert append(prob, None, lib.rope(24, table=GOOD, table_rows=9), cache) == 2
    assert append(prob, None, None, cache, total_tokens=0) == 0
    assert append(lib.problem(0, 8, 2, 64, 16, 8, 32), None, None, cache) == 0


def test_read_refusals():
    prob = lib.problem(4, 8, 2, 64, 16, 8, 32)
    cache = lib.quant_cache(GOOD, GOOD, GOOD, GOOD)
    good = [cache, GOOD, 10, GOOD, GOOD, GOOD, GOOD]
    status = lambda a: lib.status_of(lib.pa_read_quant, prob, *a)  # noqa: E731
    if not torch().cuda.is_available():
        assert status(good) in (5, 6)
    for i, bad, want in [(0, None, 1), (1, None, 1), (2, -1, 1), (2, 1 << 31, 1), (3, None, 1),
                         (4, None, 1), (1, GOOD + 2, 3), (5, GOOD + 8, 3), (6, GOOD + 2, 3)]:
        a = list(good)
        a[i] = bad
        assert status(a) == want, (i, bad)
    assert status(good[:5] + [None, None]) == 1
    assert status(good[:2] + [0] + good[3:5] + [None, None]) == 0
