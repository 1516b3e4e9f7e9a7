"""ctypes binding of libpagedattn (``include/pagedattn.h``): argument marshalling only.

Every function here forwards to the C entry point of the same name; all compute runs in
the library's CUDA kernels. Tensor arguments may be torch CUDA tensors or raw device
addresses (int). pa_append_rope, pa_decode_scored, pa_prefill_scored and the calls on a
quantised cache check the device, layout, type and length of tensors first; an address is
passed on as it is. There is no fallback: if the shared library is missing or fails to load,
``load()`` raises.
"""

from __future__ import annotations

import ctypes
import os
import sys
import threading
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libpagedattn.so")

PA_OK = 0
STATUS_NAMES = {0: "PA_OK", 1: "PA_ERR_INVALID_ARG", 2: "PA_ERR_UNSUPPORTED",
                3: "PA_ERR_MISALIGNED", 4: "PA_ERR_WORKSPACE", 5: "PA_ERR_CUDA",
                6: "PA_ERR_NO_DEVICE"}
PA_DEVERR_PAGE_ID = 1
PA_DEVERR_CONTEXT = 2
PA_DEVERR_TIMEOUT = 4
PA_DEVERR_QUERY_START = 8
PA_DEVERR_POSITION = 16
PA_TEST_EXPIRE_WAITS = 1
SCHEDULE = {"auto": 0, "single": 1, "balanced": 2}
MATH = {"auto": 0, "simt": 1, "mma": 2}
COMBINE = {"auto": 0, "fused": 1, "kernel": 2}
OUT = {"fp32": 0, "fp16": 1}
ROPE_STYLE = {"half": 0, "interleaved": 1}

# Every entry point include/pagedattn.h declares.
EXPORTS = ("pa_plan", "pa_workspace_size", "pa_workspace_init", "pa_decode", "pa_decode_ex",
           "pa_decode_noalloc", "pa_append_kv", "pa_append_rope", "pa_prefill",
           "pa_decode_scored", "pa_prefill_scored", "pa_append_quant", "pa_read_quant",
           "pa_quant_workspace_size", "pa_decode_quant", "pa_prefill_quant",
           "pa_split_kv_partial", "pa_split_kv_combine", "pa_get_device_error",
           "pa_status_string", "pa_version")


class PagedAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class pa_problem_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("query_heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages_per_sequence", ctypes.c_int32),
                ("num_physical_pages", ctypes.c_int32), ("cache_layout", ctypes.c_int32)]


class pa_options_t(ctypes.Structure):
    _fields_ = [("schedule", ctypes.c_int32), ("math", ctypes.c_int32),
                ("combine", ctypes.c_int32), ("workers", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("warps_per_cta", ctypes.c_int32),
                ("tile_tokens", ctypes.c_int32), ("test_flags", ctypes.c_int32)]


class pa_plan_t(ctypes.Structure):
    _fields_ = [("schedule", ctypes.c_int32), ("math", ctypes.c_int32),
                ("combine", ctypes.c_int32), ("workers", ctypes.c_int32),
                ("warps_per_cta", ctypes.c_int32), ("ctas", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("tile_tokens", ctypes.c_int32),
                ("units", ctypes.c_int32), ("heads_per_unit", ctypes.c_int32),
                ("group", ctypes.c_int32),
                ("smem_bytes", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64)]


class pa_rope_t(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("style", ctypes.c_int32),
                ("table_rows", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("table", ctypes.c_void_p), ("positions", ctypes.c_void_p)]
    lengths = None  # of the tensors pointed to, where rope() was given some


class pa_score_t(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("out_type", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("slopes", ctypes.c_void_p), ("first_tokens", ctypes.c_void_p),
                ("prefix_lengths", ctypes.c_void_p)]
    lengths = None  # of the tensors pointed to, where score() was given some


class pa_norm_t(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("query_weight", ctypes.c_void_p), ("key_weight", ctypes.c_void_p)]
    lengths = None  # of the tensors pointed to, where norm() was given some


class pa_quant_cache_t(ctypes.Structure):
    _fields_ = [("key", ctypes.c_void_p), ("value", ctypes.c_void_p),
                ("key_scale", ctypes.c_void_p), ("value_scale", ctypes.c_void_p)]
    lengths = None  # of the tensors pointed to, where quant_cache() was given some
    device = None   # they are on this device


_lib = None
_lock = threading.Lock()


def load(path: Optional[str] = None):
    """Load (building first if the library is absent and nvcc is available)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if path is None:
            from . import build as _build

            p = _build.build()
        lib = ctypes.CDLL(p)
        vp, i32, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
        P = ctypes.POINTER
        lib.pa_plan.argtypes = [P(pa_problem_t), P(pa_options_t), i32, P(pa_plan_t)]
        lib.pa_workspace_size.argtypes = [P(pa_problem_t), P(pa_options_t), P(ctypes.c_size_t)]
        lib.pa_workspace_init.argtypes = [vp, ctypes.c_size_t, vp]
        lib.pa_decode.argtypes = [P(pa_problem_t), vp, vp, vp, vp, vp, f32, vp, vp]
        lib.pa_decode_ex.argtypes = [P(pa_problem_t), vp, vp, vp, vp, vp, f32, vp, P(pa_options_t),
                                     vp, ctypes.c_size_t, vp]
        lib.pa_decode_noalloc.argtypes = [P(pa_problem_t), vp, vp, vp, vp, vp, f32, vp, vp]
        lib.pa_append_kv.argtypes = [P(pa_problem_t), vp, vp, vp, vp, vp, vp, vp]
        i64 = ctypes.c_int64
        lib.pa_append_rope.argtypes = [P(pa_problem_t), P(pa_rope_t), vp, i64, vp, i64, vp, i64, vp,
                                       i64, vp, vp, vp, vp, vp, vp]
        lib.pa_decode_scored.argtypes = [P(pa_problem_t), P(pa_score_t), vp, vp, vp, vp, vp, f32, vp,
                                         P(pa_options_t), vp, ctypes.c_size_t, vp]
        lib.pa_prefill_scored.argtypes = [P(pa_problem_t), P(pa_score_t), vp, vp, i64, i32, vp, vp,
                                          vp, vp, f32, vp, P(pa_options_t), vp]
        lib.pa_append_quant.argtypes = [P(pa_problem_t), P(pa_norm_t), P(pa_rope_t), vp, i64, vp, i64,
                                        vp, i64, vp, i64, vp, vp, vp, P(pa_quant_cache_t), vp]
        lib.pa_read_quant.argtypes = [P(pa_problem_t), P(pa_quant_cache_t), vp, i64, vp, vp, vp, vp,
                                      vp]
        lib.pa_quant_workspace_size.argtypes = [P(pa_problem_t), P(pa_options_t),
                                                P(ctypes.c_size_t)]
        lib.pa_decode_quant.argtypes = [P(pa_problem_t), P(pa_score_t), vp, P(pa_quant_cache_t), vp,
                                        vp, f32, vp, P(pa_options_t), vp, ctypes.c_size_t, vp]
        lib.pa_prefill_quant.argtypes = [P(pa_problem_t), P(pa_score_t), vp, vp, i64, i32,
                                         P(pa_quant_cache_t), vp, vp, f32, vp, P(pa_options_t), vp]
        lib.pa_prefill.argtypes = [P(pa_problem_t), vp, vp, ctypes.c_int64, i32, vp, vp, vp, vp,
                                   f32, vp, P(pa_options_t), vp]
        lib.pa_split_kv_partial.argtypes = [P(pa_problem_t), vp, vp, vp, vp, vp, f32, i32, i32, vp,
                                            vp, vp, vp]
        lib.pa_split_kv_combine.argtypes = [P(pa_problem_t), i32, vp, vp, vp, vp, vp]
        lib.pa_get_device_error.argtypes = [vp, P(ctypes.c_uint32)]
        lib.pa_status_string.argtypes = [ctypes.c_int]
        lib.pa_status_string.restype = ctypes.c_char_p
        lib.pa_version.argtypes = []
        for name in EXPORTS:
            if name not in ("pa_status_string",):
                getattr(lib, name).restype = ctypes.c_int
        if path is None:
            _lib = lib
        return lib


# ------------------------------------------------------------------ marshalling helpers
def problem(batch, query_heads, kv_heads, head_dim, page_size, max_pages_per_sequence,
            num_physical_pages, cache_layout=0) -> pa_problem_t:
    return pa_problem_t(batch, query_heads, kv_heads, head_dim, page_size,
                        max_pages_per_sequence, num_physical_pages, cache_layout)


def problem_of(w) -> pa_problem_t:
    """pa_problem_t of a ``workloads.Workload`` (or any object with the same fields)."""
    return problem(w.batch, w.query_heads, w.kv_heads, w.head_dim, w.page_size,
                   w.max_pages_per_sequence, w.num_physical_pages,
                   getattr(w, "cache_layout", 0))


def options(schedule="auto", math="auto", combine="auto", workers=0, stages=0,
            warps_per_cta=0, tile_tokens=0, test_flags=0) -> pa_options_t:
    o = pa_options_t()
    o.schedule = SCHEDULE[schedule] if isinstance(schedule, str) else int(schedule)
    o.math = MATH[math] if isinstance(math, str) else int(math)
    o.combine = COMBINE[combine] if isinstance(combine, str) else int(combine)
    o.workers, o.stages, o.warps_per_cta = int(workers), int(stages), int(warps_per_cta)
    o.tile_tokens = int(tile_tokens)
    o.test_flags = int(test_flags)
    return o


def rope(rotary_dim, style="half", table=None, positions=None, table_rows=None) -> pa_rope_t:
    """pa_rope_t: the position rotation of pa_append_rope. ``table`` is fp32
    [table_rows][2][rotary_dim / 2] (cosines, sines); ``positions`` int32, one per row, or None
    for the token indices. The struct keeps the tensors it points to."""
    r = pa_rope_t()
    r.rotary_dim = int(rotary_dim)
    r.style = ROPE_STYLE[style] if isinstance(style, str) else int(style)
    dev = _device()
    r.table, r.positions = _addresses("rope", dev, (table, _F32, 0), (positions, _I32, 0))
    rows = 0
    if table is not None and not isinstance(table, int):
        rows = table.shape[0]
        if r.rotary_dim != 0 and (tuple(table.shape[1:]) != (2, r.rotary_dim // 2)
                                  or (table_rows or 0) > rows):
            raise PagedAttnError(1, "rope")
    r.table_rows = int(rows if table_rows is None else table_rows)
    r.keep = (table, positions)
    r.lengths = _lengths(positions) if r.rotary_dim != 0 else None
    return r


def score(softcap=0.0, window=0, slopes=None, first_tokens=None, prefix_lengths=None,
          out="fp32") -> pa_score_t:
    """pa_score_t: the score rule of pa_decode_scored and pa_prefill_scored. ``slopes`` is fp32
    [query_heads], ``first_tokens`` int32 [query rows], ``prefix_lengths`` int32 [batch]. The
    struct keeps the tensors it points to."""
    s = pa_score_t()
    s.softcap, s.window = float(softcap), int(window)
    s.out_type = OUT[out] if isinstance(out, str) else int(out)
    dev = _device()
    s.slopes, s.first_tokens, s.prefix_lengths = _addresses(
        "score", dev, (slopes, _F32, 0), (first_tokens, _I32, 0), (prefix_lengths, _I32, 0))
    s.keep = (slopes, first_tokens, prefix_lengths)
    s.lengths = _lengths(slopes, first_tokens, prefix_lengths)
    return s


def norm(eps=1e-6, query_weight=None, key_weight=None) -> pa_norm_t:
    """pa_norm_t: the norm of queries and keys in pa_append_quant. Weights are fp32 [head_dim], or
    None: those rows are not normed. The struct keeps the tensors it points to."""
    n = pa_norm_t()
    n.eps = float(eps)
    n.query_weight, n.key_weight = _addresses("norm", _device(), (query_weight, _F32, 0),
                                              (key_weight, _F32, 0))
    n.keep = (query_weight, key_weight)
    n.lengths = _lengths(query_weight, key_weight)
    return n


def quant_cache(key, value, key_scale, value_scale) -> pa_quant_cache_t:
    """pa_quant_cache_t: codes in the problem's layout (uint8 or float8_e4m3fn tensors) and scale
    bytes [num_physical_pages][kv_heads][page_size] (uint8 or float8_e8m0fnu). The struct keeps
    the tensors it points to."""
    c = pa_quant_cache_t()
    dev = _device()
    for x in (key, value, key_scale, value_scale):
        if x is not None and not isinstance(x, int) and x.element_size() != 1:
            raise PagedAttnError(1, "quant_cache")
    c.key, c.value, c.key_scale, c.value_scale = _addresses(
        "quant_cache", dev, (key, None, 0), (value, None, 0), (key_scale, None, 0),
        (value_scale, None, 0))
    c.keep = (key, value, key_scale, value_scale)
    c.lengths = _lengths(*c.keep)
    c.device = dev
    return c


def _check_quant_cache(where, cache, prob, dev):
    """Whether the tensors of quant_cache() hold the problem's cache, on the call's device."""
    if cache is not None and cache.lengths:
        rows = prob.num_physical_pages * prob.page_size * prob.kv_heads
        n = rows * prob.head_dim
        if cache.device != dev:
            raise PagedAttnError(1, where)
        _check_lengths(where, cache, n, n, rows, rows)


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = _get_device = None  # torch's raw accessors, once the process uses a GPU


def _torch_on_gpu() -> bool:
    """Whether the process uses torch on a GPU: then there is a current device and stream, read
    through torch's raw accessors (building the stream object costs more than a small launch)."""
    global _raw_stream, _get_device
    if _raw_stream is not None:
        return True
    t = sys.modules.get("torch")
    if t is None or not t.cuda.is_initialized():
        return False
    _get_device = t._C._cuda_getDevice
    _raw_stream = t._C._cuda_getCurrentRawStream
    return True


_F16 = _F32 = _I32 = None  # torch's types, once a call may take tensors


def _device() -> int:
    """The device that a call's tensors must be on; torch's types are known from here on."""
    global _F16, _F32, _I32
    if _F16 is None and "torch" in sys.modules:
        t = sys.modules["torch"]
        _F16, _F32, _I32 = t.float16, t.float32, t.int32
    return _get_device() if _raw_stream is not None or _torch_on_gpu() else 0


def _addresses(where, dev, *args):
    """Addresses of tensor arguments (tensor, its type, the least number of its elements; a type of
    None: of its bytes), which must be whole and on device `dev`. An address passes unseen."""
    out = []
    for x, kind, least in args:
        if x is not None and x.__class__ is not int:
            if (x.get_device() != dev or not x.is_contiguous()
                    or (x.nbytes < least if kind is None
                        else x.dtype is not kind or x.numel() < least)):
                raise PagedAttnError(1, where)
            x = x.data_ptr()
        out.append(x)
    return out


def _lengths(*xs):
    """Element counts of the tensors a struct points to (None: absent, or an address), or None if
    there is none."""
    n = tuple(None if x is None or isinstance(x, int) else x.numel() for x in xs)
    return None if n.count(None) == len(n) else n


def _check_lengths(where, struct, *least):
    """Whether the tensors of rope() or score() have the elements that a call reads."""
    for have, need in zip(struct.lengths, least):
        if have is not None and have < need:
            raise PagedAttnError(1, where)


def _rows(where, dev, x, tokens, heads, head_dim, stride):
    """(address, row stride in elements) of [tokens][heads][head_dim] rows whose tokens may be
    apart, as slices of a fused projection's output are. An address takes ``stride`` as given
    (0: packed)."""
    if x is None or x.__class__ is int:
        return x, stride
    n, h, d = x.stride()
    rows, nh, nd = x.shape
    # (the strides of an empty tensor say nothing)
    if nh != heads or nd != head_dim or (rows and (d != 1 or (h != head_dim and heads > 1))) \
            or (rows > 1 and n < heads * head_dim) or rows < tokens or x.dtype is not _F16 \
            or x.get_device() != dev:
        raise PagedAttnError(1, where)
    # one row has no next one: any stride says the same
    return x.data_ptr(), n if rows > 1 else 0


def _stream(s, dev=None):
    """The stream's handle; None: torch's current stream (the default one without torch), of the
    current device, which is `dev` where the caller knows it."""
    if s is None:
        if not _torch_on_gpu():
            return None
        return _raw_stream(_get_device() if dev is None else dev)
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc: int, where: str):
    if rc != PA_OK:
        raise PagedAttnError(rc, where)


# ------------------------------------------------------------------ entry points
def pa_plan(prob: pa_problem_t, opts: Optional[pa_options_t] = None, sm_count: int = 152) -> dict:
    plan = pa_plan_t()
    _check(load().pa_plan(ctypes.byref(prob), ctypes.byref(opts) if opts else None,
                          int(sm_count), ctypes.byref(plan)), "pa_plan")
    return {name: getattr(plan, name) for name, _ in pa_plan_t._fields_}


def pa_workspace_size(prob: pa_problem_t, opts: Optional[pa_options_t] = None) -> int:
    n = ctypes.c_size_t(0)
    _check(load().pa_workspace_size(ctypes.byref(prob), ctypes.byref(opts) if opts else None,
                                    ctypes.byref(n)), "pa_workspace_size")
    return int(n.value)


def pa_workspace_init(workspace, workspace_bytes: int, stream=None):
    _check(load().pa_workspace_init(_ptr(workspace), int(workspace_bytes), _stream(stream)),
           "pa_workspace_init")


def pa_decode(prob, query, key_cache, value_cache, block_tables, context_lengths, scale, out,
              stream=None):
    _check(load().pa_decode(ctypes.byref(prob), _ptr(query), _ptr(key_cache), _ptr(value_cache),
                            _ptr(block_tables), _ptr(context_lengths), float(scale), _ptr(out),
                            _stream(stream)), "pa_decode")


def pa_decode_ex(prob, query, key_cache, value_cache, block_tables, context_lengths, scale, out,
                 opts: Optional[pa_options_t] = None, workspace=None, workspace_bytes: int = 0,
                 stream=None):
    _check(load().pa_decode_ex(ctypes.byref(prob), _ptr(query), _ptr(key_cache),
                               _ptr(value_cache), _ptr(block_tables), _ptr(context_lengths),
                               float(scale), _ptr(out), ctypes.byref(opts) if opts else None,
                               _ptr(workspace), int(workspace_bytes), _stream(stream)),
           "pa_decode_ex")


def pa_decode_noalloc(prob, query, key_cache, value_cache, block_tables, context_lengths, scale,
                      out, stream=None):
    """pa_decode without any device allocation: split-K scratch comes from a fixed 16 MiB
    array inside the library (for callers that may not allocate; see the header)."""
    _check(load().pa_decode_noalloc(ctypes.byref(prob), _ptr(query), _ptr(key_cache),
                                    _ptr(value_cache), _ptr(block_tables), _ptr(context_lengths),
                                    float(scale), _ptr(out), _stream(stream)), "pa_decode_noalloc")


PA_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


def pa_append_kv(prob, new_key, new_value, block_tables, context_lengths, key_cache, value_cache,
                 stream=None):
    """Write one new K/V row per (sequence, K/V head) at token index context_lengths[b]."""
    _check(load().pa_append_kv(ctypes.byref(prob), _ptr(new_key), _ptr(new_value),
                               _ptr(block_tables), _ptr(context_lengths), _ptr(key_cache),
                               _ptr(value_cache), _stream(stream)), "pa_append_kv")


def pa_append_rope(prob, rope, query, new_key, new_value, query_start, total_tokens, block_tables,
                   context_lengths, query_out, key_cache, value_cache, query_stride=0,
                   key_stride=0, value_stride=0, stream=None):
    """Write each sequence's last n_b tokens (rows query_start[b] .. query_start[b + 1]) into the
    caches, keys turned by position, and their turned queries into query_out. query, new_key and
    new_value may be slices of one fused projection's output (their row strides are taken from
    the tensors); query and query_out may both be None."""
    where, heads, kv_heads, hd = "pa_append_rope", prob.query_heads, prob.kv_heads, prob.head_dim
    dev = _device()
    q, qs = _rows(where, dev, query, total_tokens, heads, hd, query_stride)
    k, ks = _rows(where, dev, new_key, total_tokens, kv_heads, hd, key_stride)
    v, vs = _rows(where, dev, new_value, total_tokens, kv_heads, hd, value_stride)
    if rope is not None and rope.lengths:
        _check_lengths(where, rope, total_tokens)
    batch, cache = prob.batch, prob.num_physical_pages * prob.page_size * kv_heads * hd
    starts, bt, ctx, q_out, kc, vc = _addresses(
        where, dev, (query_start, _I32, batch + 1),
        (block_tables, _I32, batch * prob.max_pages_per_sequence), (context_lengths, _I32, batch),
        (query_out, _F16, total_tokens * heads * hd), (key_cache, _F16, cache),
        (value_cache, _F16, cache))
    _check(load().pa_append_rope(prob, rope, q, qs, k, ks, v, vs, starts, total_tokens, bt, ctx,
                                 q_out, kc, vc, _stream(stream, dev)), where)


def pa_prefill(prob, query, query_start, total_tokens, max_query_len, key_cache, value_cache,
               block_tables, context_lengths, scale, out, opts: Optional[pa_options_t] = None,
               stream=None):
    """Causal attention of each sequence's last n_b tokens (query rows query_start[b] ..
    query_start[b + 1]) over its paged cache; fp32 out [total_tokens][query_heads][head_dim]."""
    _check(load().pa_prefill(ctypes.byref(prob), _ptr(query), _ptr(query_start),
                             int(total_tokens), int(max_query_len), _ptr(key_cache),
                             _ptr(value_cache), _ptr(block_tables), _ptr(context_lengths),
                             float(scale), _ptr(out),
                             ctypes.byref(opts) if opts is not None else None,
                             _stream(stream)), "pa_prefill")


def pa_decode_scored(prob, score, query, key_cache, value_cache, block_tables, context_lengths,
                     scale, out, opts: Optional[pa_options_t] = None, workspace=None,
                     workspace_bytes: int = 0, stream=None):
    """A decode step under a score rule (``score()`` or None); out fp32 or fp16 as the rule says.
    The workspace (pa_workspace_size) needs no initialisation."""
    where, batch, heads, hd = "pa_decode_scored", prob.batch, prob.query_heads, prob.head_dim
    dev, half = _device(), False
    if score is not None:
        if score.lengths:
            _check_lengths(where, score, heads, batch)
        half = score.out_type == OUT["fp16"]
    rows, cache = batch * heads * hd, prob.num_physical_pages * prob.page_size * prob.kv_heads * hd
    q, k, v, bt, ctx, o, ws = _addresses(
        where, dev, (query, _F16, rows), (key_cache, _F16, cache), (value_cache, _F16, cache),
        (block_tables, _I32, batch * prob.max_pages_per_sequence), (context_lengths, _I32, batch),
        (out, _F16 if half else _F32, rows), (workspace, None, workspace_bytes))
    _check(load().pa_decode_scored(prob, score, q, k, v, bt, ctx, scale, o, opts, ws,
                                   workspace_bytes, _stream(stream, dev)), where)


def pa_prefill_scored(prob, score, query, query_start, total_tokens, max_query_len, key_cache,
                      value_cache, block_tables, context_lengths, scale, out,
                      opts: Optional[pa_options_t] = None, stream=None):
    """pa_prefill under a score rule (``score(out="fp16", ...)``); fp16 out."""
    where, batch, heads, hd = "pa_prefill_scored", prob.batch, prob.query_heads, prob.head_dim
    dev = _device()
    if score is not None and score.lengths:
        _check_lengths(where, score, heads, total_tokens, batch)
    rows = total_tokens * heads * hd
    cache = prob.num_physical_pages * prob.page_size * prob.kv_heads * hd
    q, qs, k, v, bt, ctx, o = _addresses(
        where, dev, (query, _F16, rows), (query_start, _I32, batch + 1), (key_cache, _F16, cache),
        (value_cache, _F16, cache), (block_tables, _I32, batch * prob.max_pages_per_sequence),
        (context_lengths, _I32, batch), (out, _F16, rows))
    _check(load().pa_prefill_scored(prob, score, q, qs, total_tokens, max_query_len, k, v, bt, ctx,
                                    scale, o, opts, _stream(stream, dev)), where)


def pa_append_quant(prob, norm, rope, query, new_key, new_value, query_start, total_tokens,
                    block_tables, context_lengths, query_out, cache, query_stride=0, key_stride=0,
                    value_stride=0, stream=None):
    """pa_append_rope into a quantised cache (``quant_cache()``), with queries and keys normed head
    by head first (``norm()`` or None)."""
    where, heads, kv_heads, hd = "pa_append_quant", prob.query_heads, prob.kv_heads, prob.head_dim
    dev = _device()
    q, qs = _rows(where, dev, query, total_tokens, heads, hd, query_stride)
    k, ks = _rows(where, dev, new_key, total_tokens, kv_heads, hd, key_stride)
    v, vs = _rows(where, dev, new_value, total_tokens, kv_heads, hd, value_stride)
    if rope is not None and rope.lengths:
        _check_lengths(where, rope, total_tokens)
    if norm is not None and norm.lengths:
        _check_lengths(where, norm, hd, hd)
    _check_quant_cache(where, cache, prob, dev)
    batch = prob.batch
    starts, bt, ctx, q_out = _addresses(
        where, dev, (query_start, _I32, batch + 1),
        (block_tables, _I32, batch * prob.max_pages_per_sequence), (context_lengths, _I32, batch),
        (query_out, _F16, total_tokens * heads * hd))
    _check(load().pa_append_quant(prob, norm, rope, q, qs, k, ks, v, vs, starts, total_tokens, bt,
                                  ctx, q_out, cache, _stream(stream, dev)), where)


def pa_read_quant(prob, cache, query_start, total_tokens, block_tables, context_lengths, key_out,
                  value_out, stream=None):
    """Each sequence's last n_b tokens of a quantised cache as fp16 rows [total_tokens][kv_heads]
    [head_dim]; key_out or value_out may be None."""
    where, batch, dev = "pa_read_quant", prob.batch, _device()
    _check_quant_cache(where, cache, prob, dev)
    rows = total_tokens * prob.kv_heads * prob.head_dim
    starts, bt, ctx, k, v = _addresses(
        where, dev, (query_start, _I32, batch + 1),
        (block_tables, _I32, batch * prob.max_pages_per_sequence), (context_lengths, _I32, batch),
        (key_out, _F16, rows), (value_out, _F16, rows))
    _check(load().pa_read_quant(prob, cache, starts, total_tokens, bt, ctx, k, v,
                                _stream(stream, dev)), where)


def pa_quant_workspace_size(prob: pa_problem_t, opts: Optional[pa_options_t] = None) -> int:
    n = ctypes.c_size_t(0)
    _check(load().pa_quant_workspace_size(prob, opts, ctypes.byref(n)), "pa_quant_workspace_size")
    return int(n.value)


def pa_decode_quant(prob, score, query, cache, block_tables, context_lengths, scale, out,
                    opts: Optional[pa_options_t] = None, workspace=None, workspace_bytes: int = 0,
                    stream=None):
    """pa_decode_scored over a quantised cache; the workspace is pa_quant_workspace_size's."""
    where, batch, heads, hd = "pa_decode_quant", prob.batch, prob.query_heads, prob.head_dim
    dev, half = _device(), False
    if score is not None:
        if score.lengths:
            _check_lengths(where, score, heads, batch)
        half = score.out_type == OUT["fp16"]
    _check_quant_cache(where, cache, prob, dev)
    rows = batch * heads * hd
    q, bt, ctx, o, ws = _addresses(
        where, dev, (query, _F16, rows),
        (block_tables, _I32, batch * prob.max_pages_per_sequence), (context_lengths, _I32, batch),
        (out, _F16 if half else _F32, rows), (workspace, None, workspace_bytes))
    _check(load().pa_decode_quant(prob, score, q, cache, bt, ctx, scale, o, opts, ws,
                                  workspace_bytes, _stream(stream, dev)), where)


def pa_prefill_quant(prob, score, query, query_start, total_tokens, max_query_len, cache,
                     block_tables, context_lengths, scale, out,
                     opts: Optional[pa_options_t] = None, stream=None):
    """pa_prefill_scored over a quantised cache; fp16 out."""
    where, batch, heads, hd = "pa_prefill_quant", prob.batch, prob.query_heads, prob.head_dim
    dev = _device()
    if score is not None and score.lengths:
        _check_lengths(where, score, heads, total_tokens, batch)
    _check_quant_cache(where, cache, prob, dev)
    rows = total_tokens * heads * hd
    q, qs, bt, ctx, o = _addresses(
        where, dev, (query, _F16, rows), (query_start, _I32, batch + 1),
        (block_tables, _I32, batch * prob.max_pages_per_sequence), (context_lengths, _I32, batch),
        (out, _F16, rows))
    _check(load().pa_prefill_quant(prob, score, q, qs, total_tokens, max_query_len, cache, bt, ctx,
                                   scale, o, opts, _stream(stream, dev)), where)


def pa_split_kv_partial(prob, query, key_cache, value_cache, block_tables, context_lengths, scale,
                        num_splits, partial_max, partial_sum, partial_out, math="auto",
                        stream=None):
    m = MATH[math] if isinstance(math, str) else int(math)
    _check(load().pa_split_kv_partial(ctypes.byref(prob), _ptr(query), _ptr(key_cache),
                                      _ptr(value_cache), _ptr(block_tables),
                                      _ptr(context_lengths), float(scale), int(num_splits), m,
                                      _ptr(partial_max), _ptr(partial_sum), _ptr(partial_out),
                                      _stream(stream)), "pa_split_kv_partial")


def pa_split_kv_combine(prob, num_splits, partial_max, partial_sum, partial_out, out, stream=None):
    _check(load().pa_split_kv_combine(ctypes.byref(prob), int(num_splits), _ptr(partial_max),
                                      _ptr(partial_sum), _ptr(partial_out), _ptr(out),
                                      _stream(stream)), "pa_split_kv_combine")


def pa_get_device_error(stream=None) -> int:
    flags = ctypes.c_uint32(0)
    _check(load().pa_get_device_error(_stream(stream), ctypes.byref(flags)),
           "pa_get_device_error")
    return int(flags.value)


def pa_status_string(status: int) -> str:
    return load().pa_status_string(int(status)).decode()


def pa_version() -> int:
    return int(load().pa_version())


def status_of(fn, *args, **kw) -> int:
    """Call a binding and return the C status instead of raising (for tests)."""
    try:
        fn(*args, **kw)
    except PagedAttnError as e:
        return e.status
    return PA_OK
