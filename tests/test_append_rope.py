"""pa_append_rope (several new tokens per sequence written to the paged caches, keys and queries
turned by position) against the formula in 64 bits; refusals on the host."""

import numpy as np
import pytest

from paged_kv_cache_63_gb300 import lib
from tests.gpu_util import torch

gpu = pytest.mark.gpu
GOOD = 1 << 20  # an aligned address that no refused call dereferences


def table_of(rows, rotary, base=10000.0):
    angle = np.arange(rows)[:, None] * base ** (-np.arange(rotary // 2) / max(1, rotary // 2))
    return np.stack([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


class Case:
    """One call's inputs on the host; every cache slot and output row starts out random."""

    def __init__(self, new, ctx, qh=8, kvh=2, hd=64, ps=16, head_major=0, rotary=None,
                 interleaved=False, explicit=False, pad=0, fused=True, seed=0, maxp=None):
        rng = np.random.default_rng(seed)
        self.new, self.ctx = np.asarray(new), np.asarray(ctx, dtype=np.int32)
        self.qh, self.kvh, self.hd, self.ps = qh, kvh, hd, ps
        self.head_major, self.interleaved, self.fused = head_major, interleaved, fused
        self.rotary = hd if rotary is None else rotary
        need = -(-self.ctx.clip(min=0) // ps)
        self.maxp = maxp or max(1, int(need.max(initial=0)))
        self.pages = int(need.sum()) + 2
        perm = rng.permutation(self.pages)
        self.bt = np.full((len(self.ctx), self.maxp), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.bt[b, :n] = perm[at:at + n]
            at += n
        self.qs = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.total = int(self.qs[-1]) + pad
        f16 = lambda *s: rng.standard_normal(s).astype(np.float16)  # noqa: E731
        self.qkv = f16(self.total, qh + 2 * kvh, hd)
        shape = (self.pages, kvh, ps, hd) if head_major else (self.pages, ps, kvh, hd)
        self.k, self.v, self.q_out = f16(*shape), f16(*shape), f16(self.total, qh, hd)
        rows = max(1, int(self.ctx.max(initial=1)))
        self.table = table_of(rows, self.rotary)
        self.positions = (rng.integers(0, rows, self.total).astype(np.int32) if explicit else None)

    def prob(self):
        return lib.problem(len(self.ctx), self.qh, self.kvh, self.hd, self.ps, self.maxp, self.pages,
                           self.head_major)

    def turned(self, rows, pos):
        """Query and key heads of `rows` turned to `pos`, in 64 bits, and the bound of the kernel's
        error: half a step of fp16, and fp32 products and sums of the pair before it."""
        x = self.qkv[rows, :self.qh + self.kvh].astype(np.float64)
        out, slack = x.copy(), np.zeros_like(x)
        r = self.rotary
        if r:
            i = np.arange(0, r, 2) if self.interleaved else np.arange(r // 2)
            j = i + (1 if self.interleaved else r // 2)
            c, s = (self.table[pos, k].astype(np.float64)[:, None] for k in (0, 1))
            out[..., i] = x[..., i] * c - x[..., j] * s
            out[..., j] = x[..., i] * s + x[..., j] * c
            both = (np.abs(x[..., i]) + np.abs(x[..., j])) * 2.0 ** -23  # two products, one sum
            slack[..., i] = slack[..., j] = both
            slack[..., :r] += np.abs(out[..., :r]) * 2.0 ** -11 + 2.0 ** -25  # and subnormals
        return out, slack

    def expected(self, skip=()):
        """(query_out, k, v) in 64 bits with their bounds (0 where values are copied)."""
        got = [a.astype(np.float64) for a in (self.q_out, self.k, self.v)]
        tol = [np.zeros_like(a) for a in got]
        for b, n in enumerate(self.new):
            for j in range(int(n)):
                row, t = int(self.qs[b]) + j, int(self.ctx[b] - n + j)
                if row in skip:
                    continue
                pos = int(self.positions[row]) if self.positions is not None else t
                x, slack = self.turned([row], [pos])
                page, slot = int(self.bt[b, t // self.ps]), t % self.ps
                at = (page, slice(None), slot) if self.head_major else (page, slot)
                got[0][row], tol[0][row] = x[0, :self.qh], slack[0, :self.qh]
                got[1][at], tol[1][at] = x[0, self.qh:], slack[0, self.qh:]
                got[2][at] = self.qkv[row, self.qh + self.kvh:]
        return got, tol

    def run(self, stream=None, with_query=True, in_place=False, **changed):
        """The call; `changed` replaces host arrays. Returns (query_out, k, v) and the flags."""
        t = torch()
        h = {n: getattr(self, n) for n in ("qkv", "qs", "bt", "ctx", "q_out", "k", "v", "table",
                                           "positions")}
        h.update(changed)
        d = {n: None if a is None else t.from_numpy(np.ascontiguousarray(a)).cuda()
             for n, a in h.items()}
        qh, kvh = self.qh, self.kvh
        parts = [d["qkv"][:, :qh], d["qkv"][:, qh:qh + kvh], d["qkv"][:, qh + kvh:]]
        if not self.fused:
            parts = [p.contiguous() for p in parts]
        q_out = parts[0] if in_place else d["q_out"]
        rope = lib.rope(self.rotary, "interleaved" if self.interleaved else "half", d["table"],
                        d["positions"])
        lib.pa_append_rope(self.prob(), rope, parts[0] if with_query else None, parts[1], parts[2],
                           d["qs"], self.total, d["bt"], d["ctx"], q_out if with_query else None,
                           d["k"], d["v"], stream=stream)
        t.cuda.synchronize()
        return [x.cpu().numpy() for x in (q_out, d["k"], d["v"])], lib.pa_get_device_error()


def check(case, got, flags=0, want_flags=0, skip=()):
    assert flags == want_flags
    for name, x, e, tol in zip(("query", "key", "value"), got, *case.expected(skip)):
        err = np.abs(x.astype(np.float64) - e)
        assert (err <= tol).all(), f"{name}: {int((err > tol).sum())} of {err.size}, {err.max()}"


CASES = {
    "one_token_each": dict(new=[1, 1, 1], ctx=[1, 16, 37]),
    "one_sequence_one_token": dict(new=[1], ctx=[1]),
    "ragged_with_empty": dict(new=[5, 0, 17, 1, 0, 40], ctx=[5, 9, 50, 1, 0, 77], pad=3),
    "empty_first_and_last": dict(new=[0, 0, 3, 0], ctx=[4, 0, 3, 2]),
    "packed_rows": dict(new=[4, 9], ctx=[20, 9], fused=False),
    "interleaved": dict(new=[6, 2], ctx=[33, 2], interleaved=True),
    "partial": dict(new=[6, 2], ctx=[33, 2], hd=128, rotary=48),
    "partial_interleaved": dict(new=[6, 2], ctx=[33, 2], hd=128, rotary=16, interleaved=True),
    "unrotated": dict(new=[6, 2], ctx=[33, 2], hd=128, rotary=0),
    "explicit_positions": dict(new=[6, 12], ctx=[33, 12], explicit=True),
    "hd128_many_heads": dict(new=[3, 1], ctx=[300, 2], qh=64, kvh=8, hd=128, ps=32),
    "hd256": dict(new=[3, 7], ctx=[130, 7], qh=24, kvh=4, hd=256, ps=64, rotary=64,
                  interleaved=True),
    "one_kv_head": dict(new=[3, 7], ctx=[130, 7], qh=7, kvh=1, hd=64, ps=8),
    "mha": dict(new=[2, 2], ctx=[20, 2], qh=40, kvh=40, hd=128),
    "many_sequences": dict(new=[1] * 1100, ctx=list(range(1, 1101)), qh=2, kvh=1, ps=256),
}


@gpu
@pytest.mark.parametrize("head_major", [0, 1])
@pytest.mark.parametrize("name", sorted(CASES))
def test_matches_formula(name, head_major):
    case = Case(head_major=head_major, **CASES[name])
    check(case, *case.run())


@gpu
def test_random_ragged_batches():
    rng = np.random.default_rng(7)
    for trial in range(12):
        n = int(rng.integers(1, 40))
        ctx = rng.integers(0, 200, n)
        new = np.minimum(ctx, rng.integers(0, 30, n) * (rng.random(n) < 0.7))
        if new.sum() == 0:
            ctx[0] = new[0] = 1
        hd = int(rng.choice([64, 128, 256]))
        case = Case(new, ctx, *[(4, 2), (6, 3), (16, 2)][trial % 3], hd=hd,
                    ps=int(rng.choice([8, 16, 64])), head_major=trial % 2,
                    rotary=int(rng.choice([0, 16, 32, hd])), interleaved=bool(trial % 3 == 1),
                    explicit=bool(trial % 4 == 2), pad=trial % 5, seed=trial)
        check(case, *case.run())


@gpu
@pytest.mark.parametrize("pad", [0, 2])
def test_no_new_tokens(pad):
    """Nothing is written, from empty tensors or from rows of a padded batch alone."""
    for fused in (True, False):
        case = Case([0, 0], [40, 3], pad=pad, fused=fused)
        check(case, *case.run())


@gpu
def test_keys_and_values_alone():
    case = Case([5, 3], [40, 3])
    got, flags = case.run(with_query=False)
    want, tol = case.expected()
    assert flags == 0 and np.array_equal(got[0], case.q_out)
    for x, e, d in list(zip(got, want, tol))[1:]:
        assert (np.abs(x - e) <= d).all()


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_query_turned_in_place(interleaved):
    case = Case([5, 3, 0, 9], [40, 3, 0, 9], fused=False, interleaved=interleaved, pad=2)
    got, flags = case.run(in_place=True)
    case.q_out = np.ascontiguousarray(case.qkv[:, :case.qh])  # rows behind the last stay
    check(case, got, flags)


@gpu
def test_turns_keep_length_and_non_finite_rows_stay_alone():
    """A rotation keeps a pair's length; a NaN reaches its own pair only."""
    case = Case([9], [9], rotary=32)
    case.qkv[4, 0, 3] = np.nan
    got, _ = case.run()
    q = got[0].astype(np.float64)
    bad = np.argwhere(np.isnan(q))
    assert bad.tolist() == [[4, 0, 3], [4, 0, 19]]
    q[4], x = 0, case.qkv[:, :case.qh].astype(np.float64)
    x[4] = 0
    len_q, len_x = (np.hypot(a[..., :16], a[..., 16:32]) for a in (q, x))
    # each of the two elements is off by at most half a step
    assert (np.abs(len_q - len_x) <= 2.0 ** -11 * 1.5 * len_x + 2.0 ** -24).all()


@gpu
def test_bad_sequences_and_tokens_are_flagged_and_skipped():
    case = Case([4, 4, 4, 4, 4], [20, 30, 40, 12, 8], pad=1)
    ctx_out = case.ctx.copy()  # lengths out of range
    ctx_out[1], ctx_out[3] = -1, case.maxp * case.ps + 1
    ctx_short = case.ctx.copy()  # more new tokens than context
    ctx_short[4] = 3
    qs_past = case.qs.copy()  # the last sequence's rows run past the batch
    qs_past[-1] = case.total + 1
    for changed, flag, bad in [(dict(ctx=ctx_out), lib.PA_DEVERR_CONTEXT, (1, 3)),
                               (dict(ctx=ctx_short), lib.PA_DEVERR_QUERY_START, (4,)),
                               (dict(qs=qs_past), lib.PA_DEVERR_QUERY_START, (4,))]:
        rows = {r for b in bad for r in range(4 * b, 4 * b + 4)}
        check(case, *case.run(**changed), want_flags=flag, skip=rows)
    # a page outside the pool: its tokens are skipped, the others of the sequence written
    bt = case.bt.copy()
    bt[1, 29 // case.ps] = case.pages
    hit = {4 + j for j in range(4) if (26 + j) // case.ps == 29 // case.ps}
    check(case, *case.run(bt=bt), want_flags=lib.PA_DEVERR_PAGE_ID, skip=hit)
    # a position outside the table
    pos = np.zeros(case.total, dtype=np.int32)
    pos[2], pos[7] = -1, case.table.shape[0]
    got, flags = case.run(positions=pos)
    assert flags == lib.PA_DEVERR_POSITION
    for r in range(case.qs[-1]):
        same = np.array_equal(got[0][r], case.q_out[r])
        assert same == (r in (2, 7)), r


@gpu
def test_captured_and_replayed_with_new_inputs():
    t = torch()
    case = Case([5, 3, 1], [40, 3, 64])
    d = {n: t.from_numpy(getattr(case, n)).cuda() for n in ("qkv", "qs", "bt", "ctx", "q_out", "k",
                                                            "v", "table")}
    rope = lib.rope(case.rotary, "half", d["table"])
    call = lambda: lib.pa_append_rope(  # noqa: E731
        case.prob(), rope, d["qkv"][:, :8], d["qkv"][:, 8:10], d["qkv"][:, 10:], d["qs"], case.total,
        d["bt"], d["ctx"], d["q_out"], d["k"], d["v"])
    call()
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        call()
    for seed in (3, 4):
        case.qkv = np.random.default_rng(seed).standard_normal(case.qkv.shape).astype(np.float16)
        d["qkv"].copy_(t.from_numpy(case.qkv))
        g.replay()
        t.cuda.synchronize()
        check(case, [d[n].cpu().numpy() for n in ("q_out", "k", "v")], lib.pa_get_device_error())


def refusal_args():
    # query, its stride, key, stride, value, stride, query_start, total, bt, ctx, q_out, k, v
    return [GOOD, 0, GOOD, 0, GOOD, 0, GOOD, 10, GOOD, GOOD, GOOD + 4096, GOOD, GOOD]


def append(prob, rope, a):
    return lib.status_of(lib.pa_append_rope, prob, rope, a[0], a[2], a[4], a[6], a[7], a[8], a[9],
                         a[10], a[11], a[12], query_stride=a[1], key_stride=a[3],
                         value_stride=a[5])


def test_refusals():
    prob = lib.problem(4, 8, 2, 64, 16, 8, 32)
    rope = lib.rope(64, "half", GOOD, table_rows=128)
    no_device = () if torch().cuda.is_available() else (5, 6)
    if no_device:
        assert append(prob, rope, refusal_args()) in no_device
        assert append(prob, None, refusal_args()) in no_device
    for i, value, status in [
            (0, None, 1), (10, None, 1), (2, None, 1), (4, None, 1), (6, None, 1), (8, None, 1),
            (9, None, 1), (11, None, 1), (12, None, 1), (7, -1, 1), (7, 1 << 31, 1),
            (1, 504, 1), (3, 120, 1), (5, -128, 1), (1, 516, 3), (3, 129, 3),
            (0, GOOD + 8, 3), (2, GOOD + 2, 3), (10, GOOD + 4100, 3), (11, GOOD + 8, 3),
            (6, GOOD + 2, 3), (9, GOOD + 1, 3)]:
        a = refusal_args()
        a[i] = value
        assert append(prob, rope, a) == status, (i, value)
    # turning a strided query in place
    a = refusal_args()
    a[10], a[1] = a[0], 1024
    assert append(prob, rope, a) == 1
    for kw, status in [(dict(rotary_dim=-16), 1), (dict(rotary_dim=80), 1), (dict(rotary_dim=8), 2),
                       (dict(rotary_dim=40), 2), (dict(style=2), 1), (dict(table_rows=0), 1),
                       (dict(table=None), 1), (dict(table=GOOD + 4), 3),
                       (dict(positions=GOOD + 2), 3)]:
        args = dict(rotary_dim=64, style="half", table=GOOD, table_rows=128)
        args.update(kw)
        assert append(prob, lib.rope(**args), refusal_args()) == status, kw
    assert append(lib.problem(4, 8, 3, 64, 16, 8, 32), rope, refusal_args()) == 1
    assert append(lib.problem(4, 8, 2, 96, 16, 8, 32), rope, refusal_args()) == 2
    # nothing to do is not an error
    a = refusal_args()
    a[7] = 0
    assert append(prob, rope, a) == 0
    assert append(lib.problem(0, 8, 2, 64, 16, 8, 32), rope, refusal_args()) == 0


def test_no_rows_need_no_addresses():
    """An empty tensor's address is null."""
    prob = lib.problem(4, 8, 2, 64, 16, 8, 32)
    a = refusal_args()
    a[0] = a[2] = a[4] = a[10] = None
    assert append(prob, None, a) == 1
    a[7] = 0
    assert append(prob, None, a) == 0


def test_reserved_field_is_refused():
    rope = lib.rope(64, "half", GOOD, table_rows=128)
    rope.reserved = 1
    assert append(lib.problem(4, 8, 2, 64, 16, 8, 32), rope, refusal_args()) == 1
    rope.rotary_dim = 0
    assert append(lib.problem(4, 8, 2, 64, 16, 8, 32), rope, refusal_args()) == 1


@gpu
def test_binding_refuses_rows_that_overlap():
    """An expanded tensor's row stride is 0, which the library takes for packed rows."""
    t = torch()
    prob = lib.problem(1, 8, 2, 64, 16, 8, 32)
    a = refusal_args()
    a[7] = 0  # nothing to do, were the rows accepted
    one = t.zeros(1, 8, 64, device="cuda", dtype=t.float16)
    a[0] = one.expand(4, 8, 64)
    assert append(prob, None, a) == 1
    a[0] = t.zeros(4 * 512, device="cuda", dtype=t.float16).as_strided((4, 8, 64), (448, 64, 1))
    assert append(prob, None, a) == 1
    a[0] = one  # a single row has no next one
    a[2] = one[:, :2].expand(4, 2, 64)
    assert append(prob, None, a) == 1
    a[2] = one[:, :2]
    assert append(prob, None, a) == 0


def test_binding_refuses_tensors_it_cannot_pass():
    t = torch()
    prob = lib.problem(1, 8, 2, 64, 16, 8, 32)
    x = t.zeros(4, 12, 64, dtype=t.float16)
    a = refusal_args()
    for wrong in (x[:, :7], x[:, :8, :32], x.transpose(1, 2)):
        a[0] = wrong
        assert append(prob, None, a) == 1
    a = refusal_args()
    a[8] = t.zeros(4, 8, dtype=t.int32)  # host memory
    assert append(prob, None, a) == 1
