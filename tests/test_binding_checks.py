"""What the binding refuses of tensors whose type or length a call of pa_append_rope,
pa_decode_scored or pa_prefill_scored could not read as what it is, before any of it reaches the
library. On the host, with tensors that claim to be on the device: whatever passes ends at the
library's own check for one."""

import pytest
import torch

from paged_kv_cache_63_gb300 import lib

# where there is a device, an argument that passed would reach a kernel
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a GPU")

B, QH, KVH, HD, PS, MAXP, PAGES, TOTAL = 3, 4, 2, 64, 16, 5, 9, 7
NO_DEVICE = (5, 6)
F16, F32, I32 = torch.float16, torch.float32, torch.int32


class OnDevice:
    """A host tensor in the place of one on device 0 (its address is passed on, not read)."""

    def __init__(self, x):
        self.x = x

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 20

    def __getattr__(self, name):
        return getattr(self.x, name)


def new(shape, dtype):
    return OnDevice(torch.zeros(shape, dtype=dtype))


def prob():
    return lib.problem(B, QH, KVH, HD, PS, MAXP, PAGES)


CACHE = ((PAGES, PS, KVH, HD), F16)
COMMON = dict(key_cache=CACHE, value_cache=CACHE, block_tables=((B, MAXP), I32),
              context_lengths=((B,), I32))
ARGS = {
    "append": dict(query=((TOTAL, QH, HD), F16), new_key=((TOTAL, KVH, HD), F16),
                   new_value=((TOTAL, KVH, HD), F16), query_start=((B + 1,), I32),
                   query_out=((TOTAL, QH, HD), F16), **COMMON),
    "decode": dict(query=((B, QH, HD), F16), out=((B, QH, HD), F32),
                   workspace=((4096,), torch.uint8), **COMMON),
    "decode_fp16": dict(query=((B, QH, HD), F16), out=((B, QH, HD), F16), **COMMON),
    "prefill": dict(query=((TOTAL, QH, HD), F16), query_start=((B + 1,), I32),
                    out=((TOTAL, QH, HD), F16), **COMMON),
}


def status(call, rope=None, score=None, **tensors):
    a = {n: new(*s) for n, s in ARGS[call].items()}
    a.update(tensors)
    if call == "append":
        return lib.status_of(lib.pa_append_rope, prob(), rope, total_tokens=TOTAL, **a)
    if call == "prefill":
        return lib.status_of(lib.pa_prefill_scored, prob(), score or lib.score(out="fp16"),
                             total_tokens=TOTAL, max_query_len=TOTAL, scale=0.1, **a)
    if score is None:
        score = lib.score(out="fp16") if call == "decode_fp16" else None
    return lib.status_of(lib.pa_decode_scored, prob(), score, scale=0.1,
                         workspace_bytes=4096 if "workspace" in a else 0, **a)


@pytest.mark.parametrize("call", sorted(ARGS))
def test_what_fits_passes(call):
    assert status(call) in NO_DEVICE
    # longer is as well
    more = {n: new((s[0] + 2, *s[1:]), t) for n, (s, t) in ARGS[call].items()}
    assert status(call, **more) in NO_DEVICE


@pytest.mark.parametrize("call,name", [(c, n) for c in sorted(ARGS) for n in sorted(ARGS[c])])
def test_types_and_lengths_are_refused(call, name):
    shape, dtype = ARGS[call][name]
    if name != "workspace":  # bytes
        for wrong in (torch.bfloat16, torch.float64, torch.int64, torch.int16, torch.uint8,
                      F32 if dtype is F16 else F16):
            assert status(call, **{name: new(shape, wrong)}) == 1, wrong
    assert status(call, **{name: new((shape[0] - 1, *shape[1:]), dtype)}) == 1
    assert status(call, **{name: new((0, *shape[1:]), dtype)}) == 1


def test_rotations():
    table, positions = new((8, 2, 16), F32), new((TOTAL,), I32)
    assert status("append", lib.rope(32, "half", table, positions)) in NO_DEVICE
    assert status("append", lib.rope(32, "half", table, positions, table_rows=5)) in NO_DEVICE
    assert status("append", lib.rope(0, "half", new((8, 2, 0), F32))) in NO_DEVICE
    assert status("append", lib.rope(32, "half", 1 << 20, 1 << 20, table_rows=8)) in NO_DEVICE
    for kw in (dict(table=new((8, 2, 16), F16)), dict(table=new((8, 2, 8), F32)),
               dict(table=new((8, 32), F32)), dict(table=new((8, 1, 16), F32)),
               dict(table=table, table_rows=9),
               dict(table=table, positions=new((TOTAL,), torch.int64))):
        with pytest.raises(lib.PagedAttnError) as e:
            lib.rope(32, "half", **kw)
        assert e.value.status == 1, kw
    assert status("append", lib.rope(32, "half", table, new((TOTAL - 1,), I32))) == 1


def test_a_layer_that_does_not_rotate_may_keep_the_others_tensors():
    """With rotary_dim 0 neither the table nor the positions are read."""
    table, few = new((8, 2, 16), F32), new((TOTAL - 1,), I32)
    assert status("append", lib.rope(0, "half", table, few)) in NO_DEVICE


@pytest.mark.parametrize("call,rows", [("decode", B), ("prefill", TOTAL)])
def test_score_rules(call, rows):
    out = "fp16" if call == "prefill" else "fp32"
    fits = dict(slopes=new((QH,), F32), first_tokens=new((rows,), I32),
                prefix_lengths=new((B,), I32))
    assert status(call, score=lib.score(out=out, **fits)) in NO_DEVICE
    for name, x in fits.items():
        for wrong in (torch.int64, F16):
            with pytest.raises(lib.PagedAttnError) as e:
                lib.score(out=out, **{name: new(tuple(x.shape), wrong)})
            assert e.value.status == 1
        short = lib.score(out=out, **{name: new((x.shape[0] - 1,), x.dtype)})
        if (call, name) != ("decode", "prefix_lengths"):  # a decode step does not read them
            assert status(call, score=short) == 1, name
    own = lib.pa_score_t(out_type=lib.OUT[out], slopes=1 << 20)  # a caller's own struct
    assert status(call, score=own) in NO_DEVICE


def test_the_output_has_the_rules_type():
    assert status("decode", score=lib.score(out="fp16")) == 1
    assert status("decode_fp16", score=lib.score()) == 1
