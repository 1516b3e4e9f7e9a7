"""Calls from threads of the host."""

import threading

import pytest

from paged_kv_cache_63_gb300 import lib
from tests.gpu_util import torch
from tests.scored_reference import Cached
from tests.test_append_rope import table_of

gpu = pytest.mark.gpu


def entry_points(w):
    """Name: (call, its outputs) over the inputs of w, one new token to a sequence."""
    t = torch()
    d, prob = w.to_device(), w.prob()
    b, qh, kvh, hd = w.batch, w.query_heads, w.kv_heads, w.head_dim
    out = lambda dt=t.float32: t.zeros(b, qh, hd, dtype=dt, device="cuda")  # noqa: E731
    n = lib.pa_workspace_size(prob)
    ws = t.empty(n, dtype=t.uint8, device="cuda")
    lib.pa_workspace_init(ws, n)
    qs = t.arange(b + 1, dtype=t.int32, device="cuda")
    kv = [t.randn(b, kvh, hd, device="cuda").half() for _ in range(2)]
    caches = d["k"].clone(), d["v"].clone()
    before = d["ctx"] - 1
    rope = lib.rope(hd, "half", t.from_numpy(table_of(int(w.ctx.max()), hd)).cuda())
    score = lib.score(softcap=5.0, out="fp16")
    splits = [t.zeros(b, qh, 4, device="cuda") for _ in range(2)] + \
        [t.zeros(b, qh, 4, hd, device="cuda")]
    cached, scale = (d["k"], d["v"], d["bt"], d["ctx"]), w.scale
    half = lambda: out(t.float16)  # noqa: E731
    o = dict(decode=out(), decode_ex=out(), noalloc=out(), prefill=out(), append_rope=half(),
             decode_scored=half(), prefill_scored=half())
    return {
        "decode": (lambda: lib.pa_decode(prob, d["q"], *cached, scale, o["decode"]),
                   [o["decode"]]),
        "decode_ex": (lambda: lib.pa_decode_ex(prob, d["q"], *cached, scale, o["decode_ex"],
                                               lib.options(), ws, n), [o["decode_ex"]]),
        "decode_noalloc": (lambda: lib.pa_decode_noalloc(prob, d["q"], *cached, scale,
                                                         o["noalloc"]), [o["noalloc"]]),
        "append_kv": (lambda: lib.pa_append_kv(prob, *kv, d["bt"], before, *caches), caches),
        "append_rope": (lambda: lib.pa_append_rope(prob, rope, d["q"], *kv, qs, b, d["bt"],
                                                   d["ctx"], o["append_rope"], *caches),
                        [o["append_rope"], *caches]),
        "prefill": (lambda: lib.pa_prefill(prob, d["q"], qs, b, 1, *cached, scale, o["prefill"]),
                    [o["prefill"]]),
        "decode_scored": (lambda: lib.pa_decode_scored(prob, score, d["q"], *cached, scale,
                                                       o["decode_scored"], workspace=ws,
                                                       workspace_bytes=n), [o["decode_scored"]]),
        "prefill_scored": (lambda: lib.pa_prefill_scored(prob, score, d["q"], qs, b, 1, *cached,
                                                         scale, o["prefill_scored"]),
                           [o["prefill_scored"]]),
        "split_kv_partial": (lambda: lib.pa_split_kv_partial(prob, d["q"], *cached, scale, 4,
                                                             *splits), splits),
    }


@gpu
@pytest.mark.parametrize("head_major", [0, 1])
def test_a_threads_first_call(head_major):
    """A thread has no CUDA context of its own until some call needs one, which may be any of the
    library's."""
    t = torch()
    for name, (call, outs) in entry_points(Cached([700, 33], head_major=head_major)).items():
        call()
        t.cuda.synchronize()
        want = [x.clone() for x in outs]
        for x in outs:
            x.zero_()
        t.cuda.synchronize()
        failed = []

        def first():
            try:
                call()
            except lib.PagedAttnError as e:
                failed.append(e)

        thread = threading.Thread(target=first)
        thread.start()
        thread.join()
        t.cuda.synchronize()
        assert not failed, (name, failed)
        assert lib.pa_get_device_error() == 0
        for x, y in zip(outs, want):
            if name.startswith("append"):  # slots of no token were cleared with the others
                y = y.masked_fill(x == 0, 0)
            assert t.equal(x, y), name
