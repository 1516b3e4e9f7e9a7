"""Attention under a score rule in 64 bits, with a bound of a kernel's error derived from the
number formats it goes through, and the inputs of the tests of pa_decode_scored and
pa_prefill_scored."""

import dataclasses
from typing import Optional

import numpy as np


@dataclasses.dataclass
class Rule:
    softcap: float = 0.0
    window: int = 0
    slopes: Optional[np.ndarray] = None  # [query_heads]
    first: Optional[np.ndarray] = None   # [rows]
    prefix: Optional[np.ndarray] = None  # [batch]


def seen(rule, b, row, pos, ctx):
    """The half-open range of tokens that a row at position pos of sequence b sees."""
    lo, end = 0, pos + 1
    if rule.window:
        lo = max(lo, pos - rule.window + 1)
    if rule.first is not None:
        lo = max(lo, int(rule.first[row]))
    if rule.prefix is not None and pos < rule.prefix[b]:
        end = min(int(rule.prefix[b]), ctx)
    return lo, max(end, lo)


def attend(case, rule, probability_error, weight_floor, cap_error=2.0 ** -22, span=0):
    """(out, bound) in 64 bits over case's query rows; rows that are no new token's stay NaN.

    A kernel's weight of token t carries a relative error e_t: the dot product's accumulation
    (the products are exact in fp32; at most head_dim / 16 + 2 additions, each off by 2^-23 of
    the terms' absolute sum), the roundings of the scaled, capped and biased score (2^-22 of
    each, tanhf's two last places among them), the exponential (2^-22, and 2^-24 of its
    argument), `cap_error` of a capped score, a bias formed in two parts of up to `span` tokens
    each, and `probability_error`, the rounding of the probabilities that meet V. The
    weighted mean out = sum w v / sum w is then off by at most sum w e (|v| + |out|), plus the
    fp32 sums over the tiles (2^-24 of sum w |v| for each of n additions), plus
    `weight_floor`, the smallest weight the probability's type tells from 0, on every token."""
    w = case
    g = w.query_heads // w.kv_heads
    out = np.full((w.rows, w.query_heads, w.head_dim), np.nan)
    bound = np.zeros_like(out)
    for b in range(w.batch):
        keys, values = w.gathered(b)
        for row, pos in w.rows_of(b):
            lo, end = seen(rule, b, row, pos, int(w.ctx[b]))
            for h in range(w.query_heads):
                if end <= lo:
                    out[row, h] = 0.0
                    continue
                q = w.q[row, h].astype(np.float64)
                k = keys[lo:end, h // g].astype(np.float64)
                v = values[lo:end, h // g].astype(np.float64)
                s = w.scale * (k @ q)
                e = abs(w.scale) * (np.abs(k) @ np.abs(q)) * (w.head_dim / 16 + 2) * 2.0 ** -23
                e += np.abs(s) * 2.0 ** -22
                if rule.softcap:
                    s = rule.softcap * np.tanh(s / rule.softcap)
                    e += np.abs(s) * cap_error
                if rule.slopes is not None:
                    bias = float(rule.slopes[h]) * np.abs(pos - np.arange(lo, end))
                    s = s - bias
                    e += (np.abs(bias) + abs(float(rule.slopes[h])) * span) * 2.0 ** -22
                e += (np.abs(s) + np.abs(s.max())) * 2.0 ** -23 + 2.0 ** -22 + probability_error
                p = np.exp(s - s.max())
                p /= p.sum()
                o = p @ v
                out[row, h] = o
                n = end - lo
                bound[row, h] = ((p * e) @ np.abs(v) + (p @ e) * np.abs(o)
                                 + n * 2.0 ** -24 * (p @ np.abs(v))
                                 + weight_floor * p.max() * (np.abs(v).sum(0) + n * np.abs(o)))
    return out, bound


class Cached:
    """Queries and a paged cache on the host. Every slot and page no token of a sequence lives
    in holds NaN (K) or Inf (V), and the table's unused entries point outside the pool."""

    def __init__(self, ctx, new=None, qh=4, kvh=2, hd=64, ps=16, head_major=0, seed=0, q_scale=1.0,
                 pad=0, maxp=None, spare=1):
        rng = np.random.default_rng(seed)
        self.ctx = np.asarray(ctx, dtype=np.int32)
        self.batch, self.query_heads, self.kv_heads = len(self.ctx), qh, kvh
        self.head_dim, self.ps, self.head_major = hd, ps, head_major
        self.scale = 1.0 / np.sqrt(hd)
        self.new = None if new is None else np.asarray(new)
        need = -(-self.ctx.astype(np.int64) // ps)
        self.maxp = maxp or max(1, int(need.max(initial=0)))
        self.pages = int(need.sum()) + spare
        perm = rng.permutation(self.pages)
        self.bt = np.full((self.batch, self.maxp), self.pages + 7, dtype=np.int32)
        shape = (self.pages, ps, kvh, hd)
        self.k = np.full(shape, np.nan, dtype=np.float16)
        self.v = np.full(shape, np.inf, dtype=np.float16)
        at = 0
        for b in range(self.batch):
            n, m = int(self.ctx[b]), int(need[b])
            self.bt[b, :m] = perm[at:at + m]
            at += m
            t = np.arange(n)
            where = (self.bt[b, t // ps], t % ps)
            self.k[where] = rng.standard_normal((n, kvh, hd)).astype(np.float16)
            self.v[where] = rng.standard_normal((n, kvh, hd)).astype(np.float16)
        if self.new is None:  # a decode step
            self.rows, self.qs = self.batch, None
        else:
            self.qs = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
            self.rows = int(self.qs[-1]) + pad
        self.q = (q_scale * rng.standard_normal((self.rows, qh, hd))).astype(np.float16)

    def gathered(self, b):
        t = np.arange(int(self.ctx[b]))
        return (self.k[self.bt[b, t // self.ps], t % self.ps],
                self.v[self.bt[b, t // self.ps], t % self.ps])

    def rows_of(self, b):
        n = int(self.ctx[b])
        if self.qs is None:
            return [(b, n - 1)]
        m = int(self.new[b])
        return [(int(self.qs[b]) + j, n - m + j) for j in range(m)]

    def forget(self, b, before):
        """Sequence b's tokens before `before` leave the cache: their whole pages leave the table,
        their slots in the page that stays hold NaN and Inf."""
        for t in range(before):
            page, slot = self.bt[b, t // self.ps], t % self.ps
            self.k[page, slot] = np.nan
            self.v[page, slot] = np.inf
        self.bt[b, :before // self.ps] = -5

    def cache(self, x):
        return np.ascontiguousarray(x.transpose(0, 2, 1, 3)) if self.head_major else x

    def prob(self):
        from paged_kv_cache_63_gb300 import lib

        return lib.problem(self.batch, self.query_heads, self.kv_heads, self.head_dim, self.ps,
                           self.maxp, self.pages, self.head_major)

    def to_device(self):
        import torch as t

        put = lambda a: None if a is None else t.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return dict(q=put(self.q), k=put(self.cache(self.k)), v=put(self.cache(self.v)),
                    bt=put(self.bt), ctx=put(self.ctx), qs=put(self.qs))


def device_rule(rule, out):
    from paged_kv_cache_63_gb300 import lib
    import torch as t

    put = lambda a, dt: None if a is None else t.from_numpy(np.asarray(a, dtype=dt)).cuda()  # noqa: E731
    return lib.score(softcap=rule.softcap, window=rule.window, slopes=put(rule.slopes, np.float32),
                     first_tokens=put(rule.first, np.int32),
                     prefix_lengths=put(rule.prefix, np.int32), out=out)


def slopes_of(heads):
    return np.exp2(-8.0 * np.arange(1, heads + 1) / heads).astype(np.float32)


def assert_within(got, want, bound, half_out):
    """Every element within its bound, and half a step of fp16 where the output is rounded."""
    got = np.asarray(got, dtype=np.float64)
    live = ~np.isnan(want)
    assert np.isfinite(got[live]).all(), "non-finite output"
    err = np.abs(got - want)[live]
    tol = bound[live].copy()
    if half_out:
        tol += (np.abs(want[live]) + tol) * 2.0 ** -11 + 2.0 ** -25
    assert (err <= tol).all(), (f"{int((err > tol).sum())} of {err.size} elements out of bound; "
                                f"worst {np.max(err / np.maximum(tol, 1e-300)):.2f} times it")
    return float(np.max(err / np.maximum(tol, 1e-300), initial=0.0))
