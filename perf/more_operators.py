"""The operators of the quantised paged K/V cache: what is measured of them, and their plain forms.

The caches hold e4m3 values, one power-of-two scale (e8m0) for each token and K/V head:

* ``append``  -- ``pa_append_quant``: the newest tokens' queries, keys and values, taken from the
  fused projection's rows; queries and keys normed head by head and rotated by position, keys
  and values rounded to 8 bits as they are written into the paged caches.
* ``read``    -- ``pa_read_quant``: the newest tokens of each sequence read back as fp16 rows.
* ``decode``  -- ``pa_decode_quant``: one new token per sequence attends over the 8-bit cache.
* ``prefill`` -- ``pa_prefill_quant``: a chunk of new tokens per sequence does.

A row x of a key or value is held as codes c and a scale 2^e: e is the smallest integer of
-15 .. 8 with max |x| <= 448 * 2^e, c the e4m3 number nearest to x / 2^e (at most 448, or 240 for
e = 8, so that c * 2^e is always a finite fp16 number).

``run`` computes the plain form in elementary torch operations in 32 bits (the rows that are
rounded to 8 bits in 64: a key next to the border of two codes), or, where ``own`` is true,
makes the calls a user makes. Sizes are those of the repository's workloads (tiny, gqa4_mid, mha,
long_gqa6, ragged and the multi-token ones) and of the range around them.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BASE = 10000.0  # of the rotation's frequencies
EPS = 1e-6      # of the norm


# ------------------------------------------------------------------------------- cases
def _case(name, op, **kw):
    c = dict(op=op, batch=2, query_heads=4, kv_heads=2, head_dim=64, page_size=16,
             head_major=False, ctx_lo=1, ctx_hi=64, new_lo=1, new_hi=1, pad_rows=0, mix=1)
    if op == "append":
        c.update(rotary=64, interleaved=False, explicit=False, norm=True)
    elif op != "read":
        c.update(softcap=0.0, window=0, alibi=False, documents=0, prefix=0, half_out=True)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # ---- append
        # one decode step of a full serving batch (the ragged workload's heads): latency counts
        _case("append_step", "append", batch=256, query_heads=64, kv_heads=8, head_dim=128,
              page_size=32, ctx_lo=1, ctx_hi=1024, rotary=128, mix=1),
        # eight fresh 2048-token prompts written at once (prefill_gqa4's shape)
        _case("append_prompts", "append", batch=8, query_heads=32, kv_heads=8, head_dim=128,
              page_size=16, ctx_lo=2048, ctx_hi=2048, new_lo=2048, new_hi=2048, rotary=128, mix=2),
        # ragged chunks on cached prefixes: no norm, partial rotation of neighbouring pairs at
        # positions given by the caller, head-major pages, rows of a padded batch at the end
        _case("append_chunks", "append", batch=13, query_heads=24, kv_heads=4, head_dim=256,
              page_size=64, head_major=True, ctx_lo=512, ctx_hi=4096, new_lo=1, new_hi=509,
              pad_rows=5, rotary=64, interleaved=True, explicit=True, norm=False, mix=3),
        # ---- read
        # the last tokens of two short sequences, read back to check or move them: latency
        _case("read_tiny", "read", batch=2, ctx_lo=37, ctx_hi=100, new_lo=20, new_hi=37, mix=4),
        # a mid-size batch (gqa4_mid) moved to a cache of 16 bits
        _case("read_batch", "read", batch=32, query_heads=32, kv_heads=8, head_dim=128,
              page_size=16, ctx_lo=512, ctx_hi=4096, new_lo=4096, new_hi=4096, mix=5),
        # ---- decode
        # two short sequences: latency
        _case("decode_tiny", "decode", batch=2, ctx_lo=37, ctx_hi=100, mix=6),
        # a mid-size batch (gqa4_mid), output in 32 bits
        _case("decode_mid", "decode", batch=32, query_heads=32, kv_heads=8, head_dim=128,
              page_size=16, ctx_lo=512, ctx_hi=4096, half_out=False, mix=7),
        # every head with keys of its own (mha): a local layer's capped scores in a window
        _case("decode_mha_window", "decode", batch=64, query_heads=32, kv_heads=32, head_dim=128,
              page_size=16, ctx_lo=2048, ctx_hi=2048, softcap=50.0, window=1500, mix=8),
        # four 100k-token contexts (long_gqa6): the longest reads
        _case("decode_long", "decode", batch=4, query_heads=24, kv_heads=4, head_dim=256,
              page_size=64, ctx_lo=100000, ctx_hi=100000, mix=9),
        # ---- prefill
        # a few drafted tokens checked at once on cached contexts: little work to a read
        _case("prefill_drafts", "prefill", batch=8, query_heads=32, kv_heads=8, head_dim=128,
              page_size=16, ctx_lo=512, ctx_hi=4096, new_lo=2, new_hi=7, mix=10),
        # chunked prefill (prefill_chunked): the last 512 tokens of 16 contexts
        _case("prefill_chunked", "prefill", batch=16, query_heads=32, kv_heads=8, head_dim=128,
              page_size=16, ctx_lo=512, ctx_hi=4096, new_lo=512, new_hi=512, mix=11),
        # two 4096-token prompts (prefill_gqa6_hd256), scores capped
        _case("prefill_hd256", "prefill", batch=2, query_heads=24, kv_heads=4, head_dim=256,
              page_size=64, ctx_lo=4096, ctx_hi=4096, new_lo=4096, new_hi=4096, softcap=50.0,
              mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most, size = {}, {}
    for c in listed():
        w, op = work(c), c["op"]
        most[op] = max(most.get(op, 0.0), max(w["bytes"], w["flops"] / 100))
        size[op] = max(size.get(op, 0), _plain_size(c))
    while True:
        op = rng.choice(["append", "read", "decode", "prefill"])
        qh, kvh = rng.choice([(4, 2), (8, 1), (8, 8), (16, 2), (14, 2), (24, 4), (32, 8),
                              (32, 32), (64, 8), (40, 8), (48, 4)])
        hd = rng.choice([64, 128, 256])
        ps = rng.choice([8, 16, 32, 64, 128, 256])
        hi = _log(rng, 8, 100000 if op == "decode" else 4096)
        lo = rng.randint(0, hi) if rng.random() < 0.7 else hi
        c = dict(batch=_log(rng, 1, 256), query_heads=qh, kv_heads=kvh, head_dim=hd, page_size=ps,
                 head_major=rng.random() < 0.3, ctx_lo=lo, ctx_hi=hi, mix=rng.randrange(1 << 30))
        if op != "decode":
            top = _log(rng, 1, 4096)
            c.update(new_lo=rng.randint(0, top), new_hi=top, pad_rows=rng.choice([0, 0, 3]))
        if op == "append":
            c.update(rotary=rng.choice([0, 16, 32, 48, 64, hd, hd, hd]), norm=rng.random() < 0.6,
                     interleaved=rng.random() < 0.4, explicit=rng.random() < 0.3)
        elif op != "read":
            c.update(softcap=rng.choice([0.0, 0.0, 20.0, 30.0, 50.0]),
                     window=_log(rng, 1, 4096) if rng.random() < 0.3 else 0,
                     alibi=rng.random() < 0.2,
                     documents=_log(rng, 8, 4096) if rng.random() < 0.2 else 0,
                     half_out=op == "prefill" or rng.random() < 0.7)
            if op == "prefill" and rng.random() < 0.2:
                c["prefix"] = _log(rng, 1, 4096)
        c = _case(None, op, **c)
        w = work(c)
        if max(w["bytes"], w["flops"] / 100) <= most[op] and _plain_size(c) <= size[op] \
                and w["bytes"] > 4096:
            return c


def _plain_size(c):
    """Values that the plain form holds at once: padded scores and gathered keys."""
    if c["op"] in ("append", "read"):
        return c["batch"] * c["ctx_hi"] * c["kv_heads"] * c["head_dim"]
    rows = c["new_hi"] if c["op"] == "prefill" else 1
    return c["batch"] * c["ctx_hi"] * (c["query_heads"] * min(rows, c["ctx_hi"])
                                       + c["kv_heads"] * c["head_dim"])


# ------------------------------------------------------------------------------- geometry
def _lengths(c):
    """Context lengths (new tokens included) and new-token counts of the sequences."""
    r = random.Random(c["mix"])
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["batch"])]
    if c["op"] == "decode":
        return np.array(ctx), np.minimum(1, np.array(ctx))
    new = [min(n, r.randint(c["new_lo"], c["new_hi"])) for n in ctx]
    if sum(new) == 0:
        ctx[0] = max(ctx[0], 1)
        new[0] = 1
    return np.array(ctx), np.array(new)


def _first(c):
    """For each sequence the first token of every position's document."""
    r = random.Random(c["mix"] + 1)
    ctx, _ = _lengths(c)
    out = []
    for n in ctx:
        first, at = np.zeros(int(n), dtype=np.int64), 0
        while c.get("documents", 0) and at < n:
            first[at:] = at
            at += r.randint(1, 2 * c["documents"])
        out.append(first)
    return out


def _visible(c):
    """For each sequence the arrays lo, hi of its new tokens: token t is seen if lo <= t <= hi."""
    ctx, new = _lengths(c)
    got = []
    for first, n, m in zip(_first(c), ctx.tolist(), new.tolist()):
        p = np.arange(n - m, n)
        lo = first[p] if m else p
        if c["window"]:
            lo = np.maximum(lo, p - c["window"] + 1)
        hi = np.maximum(p, min(c["prefix"], n) - 1) if c["prefix"] else p
        hi = np.where(p < c["prefix"], hi, p)
        got.append((lo, hi))
    return got


def work(case):
    c = case
    ctx, new = _lengths(c)
    total, hd, qh, kvh = int(new.sum()), c["head_dim"], c["query_heads"], c["kv_heads"]
    table = 4.0 * (-(-ctx // c["page_size"])).sum()
    row = hd + 1.0  # a cached row: codes and a scale
    if c["op"] == "append":
        turned = total * (qh + kvh) * c["rotary"]
        normed = total * (qh + kvh) * hd if c["norm"] else 0
        angles = min(total, int(ctx.max())) * c["rotary"] * 4
        return {"bytes": total * (4.0 * qh * hd + 4.0 * kvh * hd + 2.0 * kvh * row) + angles
                + 8.0 * total, "flops": 3.0 * turned + 4.0 * normed + 4.0 * total * kvh * hd}
    if c["op"] == "read":
        return {"bytes": total * 2.0 * kvh * (row + 2.0 * hd) + 4.0 * total,
                "flops": 2.0 * total * kvh * hd}
    pairs = tokens = 0
    for lo, hi in _visible(c):
        if len(lo):
            pairs += int((hi - lo + 1).sum())
            tokens += int(hi.max() - lo.min() + 1)
    out_bytes = 2 if c["half_out"] else 4
    rows = total if c["op"] == "prefill" else c["batch"]
    return {"bytes": float(2.0 * tokens * kvh * row + rows * qh * hd * (2.0 + out_bytes) + table),
            "flops": float(4.0 * hd * qh * pairs)}


# ------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.float16)  # noqa: E731
    ints = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
    ctx, new = _lengths(c)
    B, ps, kvh, hd, qh = c["batch"], c["page_size"], c["kv_heads"], c["head_dim"], c["query_heads"]
    need = -(-ctx // ps)
    maxp, pages = max(1, int(need.max())), max(1, int(need.sum()))
    perm = np.random.RandomState(seed % (1 << 31)).permutation(pages)
    bt = np.full((B, maxp), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        bt[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    total = int(new.sum()) + c["pad_rows"]

    def cache():
        # codes as rows of normal values have them: the largest of a row lies above 224
        codes = torch.empty(pages, kvh if c["head_major"] else ps, ps if c["head_major"] else kvh,
                            hd, dtype=torch.uint8, device=DEV)
        for part in codes.split(max(1, (1 << 26) // (ps * kvh * hd))):
            part.copy_((normal(*part.shape) * 100.0).clamp(-448.0, 448.0)
                       .to(torch.float8_e4m3fn).view(torch.uint8))
        scale = torch.randint(127 - 8, 127 - 5, (pages, kvh, ps), generator=g, device=DEV,
                              dtype=torch.uint8)
        return codes, scale

    (k, ks), (v, vs) = cache(), cache()
    s = dict(case=dict(c), bt=ints(bt), ctx=ints(ctx), k=k, ks=ks, v=v, vs=vs,
             qs=ints(np.concatenate([[0], np.cumsum(new)])), total=total, maxp=maxp, pages=pages,
             scale=1.0 / math.sqrt(hd), max_ctx=int(ctx.max()), max_new=int(new.max()))
    if c["op"] == "append":
        # the fused projection's output: each token's query, key and value rows side by side; keys
        # of a few channels are larger than the rest
        s["qkv"] = normal(total, qh + 2 * kvh, hd)
        s["qkv"][:, qh:qh + kvh, ::37] *= 8.0
        s["q_out"] = normal(total, qh, hd)
        half = c["rotary"] // 2
        rows = max(1, int(ctx.max()))
        turn = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * BASE ** (
            -torch.arange(half, device=DEV, dtype=torch.float64) / max(1, half))
        s["table"] = torch.stack([turn.cos(), turn.sin()], 1).float().contiguous()
        s["positions"] = s["q_weight"] = s["k_weight"] = None
        if c["explicit"]:
            s["positions"] = torch.randint(0, rows, (total,), generator=g, device=DEV,
                                           dtype=torch.int32)
        if c["norm"]:
            s["q_weight"], s["k_weight"] = (1.0 + 0.2 * normal(hd).float() for _ in range(2))
    elif c["op"] == "read":
        s["k_out"], s["v_out"] = normal(total, kvh, hd), normal(total, kvh, hd)
    else:
        # queries a little longer than unit normals, so that some scores reach the cap
        rows = B if c["op"] == "decode" else total
        s["q"] = (normal(rows, qh, hd).float() * 3.0).half()
        s["slopes"] = None
        if c["alibi"]:
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, qh + 1, device=DEV) / qh).float()
        s["first"] = s["prefix"] = None
        if c["documents"]:
            f = [(a[n - m:] if c["op"] == "prefill" else a[-1:] if n else np.zeros(1, np.int64))
                 for a, n, m in zip(_first(c), ctx.tolist(), new.tolist())]
            f = np.concatenate(f)
            s["first"] = ints(np.concatenate([f, np.zeros(rows - len(f), np.int64)]))
        if c["prefix"]:
            s["prefix"] = ints(np.minimum(c["prefix"], ctx))
        s["out"] = torch.zeros(rows, qh, hd, device=DEV,
                               dtype=torch.float16 if c["half_out"] else torch.float32)
    if own:
        s["handle"] = _handle(s)
    return s


# ------------------------------------------------------------------------------- the framework
def _handle(s):
    """What a serving program keeps beside its tensors: the problem, the cache, the rule and a
    workspace."""
    from paged_kv_cache_63_gb300 import lib

    c = s["case"]
    prob = lib.problem(c["batch"], c["query_heads"], c["kv_heads"], c["head_dim"],
                       c["page_size"], s["maxp"], s["pages"], int(c["head_major"]))
    h = dict(lib=lib, prob=prob, cache=lib.quant_cache(s["k"], s["v"], s["ks"], s["vs"]))
    if c["op"] == "append":
        h["rope"] = lib.rope(c["rotary"], "interleaved" if c["interleaved"] else "half",
                             s["table"], s["positions"])
        h["norm"] = lib.norm(EPS, s["q_weight"], s["k_weight"]) if c["norm"] else None
    elif c["op"] != "read":
        h["score"] = lib.score(softcap=c["softcap"], window=c["window"], slopes=s["slopes"],
                               first_tokens=s["first"], prefix_lengths=s["prefix"],
                               out="fp16" if c["half_out"] else "fp32")
    if c["op"] == "decode":
        h["n"] = lib.pa_quant_workspace_size(prob)
        h["ws"] = torch.empty(max(h["n"], 256), dtype=torch.uint8, device=DEV)
    return h


def _run_own(s):
    c, h = s["case"], s["handle"]
    lib = h["lib"]
    if c["op"] == "append":
        qh, kvh = c["query_heads"], c["kv_heads"]
        qkv = s["qkv"]
        lib.pa_append_quant(h["prob"], h["norm"], h["rope"], qkv[:, :qh], qkv[:, qh:qh + kvh],
                            qkv[:, qh + kvh:], s["qs"], s["total"], s["bt"], s["ctx"],
                            s["q_out"], h["cache"])
        return _cache_values(s, s["q_out"])
    if c["op"] == "read":
        lib.pa_read_quant(h["prob"], h["cache"], s["qs"], s["total"], s["bt"], s["ctx"],
                          s["k_out"], s["v_out"])
        return {"key": s["k_out"], "value": s["v_out"]}
    if c["op"] == "decode":
        lib.pa_decode_quant(h["prob"], h["score"], s["q"], h["cache"], s["bt"], s["ctx"],
                            s["scale"], s["out"], workspace=h["ws"], workspace_bytes=h["n"])
    else:
        lib.pa_prefill_quant(h["prob"], h["score"], s["q"], s["qs"], s["total"], s["max_new"],
                             h["cache"], s["bt"], s["ctx"], s["scale"], s["out"])
    return s["out"]


# ------------------------------------------------------------------------------- plain forms
def _cache_values(s, q_out):
    """The written caches as the numbers that their bytes stand for."""
    return {"query": q_out,
            "key_cache": s["k"].view(torch.float8_e4m3fn),
            "value_cache": s["v"].view(torch.float8_e4m3fn),
            "key_scale": s["ks"].view(torch.float8_e8m0fnu),
            "value_scale": s["vs"].view(torch.float8_e8m0fnu)}


def _quantise(x):
    """(codes, scale bytes) of rows in 64 bits."""
    top = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)  # top = m * 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(top > 0, e, -15).clamp(-15, 8)
    most = torch.where(e < 8, 448.0, 240.0)
    y = torch.ldexp(x, -e)
    y = torch.minimum(torch.maximum(y, -most), most)
    # to the nearest of 4 significant bits (at least 2^-9 apart), ties to even
    _, f = torch.frexp(y)
    step = torch.exp2((f - 4).clamp(min=-9).to(x.dtype))
    y = torch.round(y / step) * step
    return y.to(torch.float8_e4m3fn).view(torch.uint8), (e[..., 0] + 127).to(torch.uint8)


def _rows_of_sequences(s):
    """For each row its sequence, its token's position, and whether it is a new token's."""
    row = torch.arange(s["total"], device=DEV)
    b = (torch.searchsorted(s["qs"].long(), row, right=True) - 1).clamp(0, s["case"]["batch"] - 1)
    qs, ctx = s["qs"].long(), s["ctx"].long()
    pos = ctx[b] - qs[b + 1] + row
    return b, pos, row < qs[-1]


def _norm(x, weight):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _turn(s, x, pos):
    """The first `rotary` elements of each head turned by position."""
    c = s["case"]
    half = c["rotary"] // 2
    if not half:
        return x
    at = s["positions"].long() if c["explicit"] else pos.clamp(min=0, max=s["max_ctx"] - 1)
    cos, sin = (s["table"][at, i][:, None, :].to(x.dtype) for i in (0, 1))
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if c["interleaved"]:
        a, d = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - d * sin, a * sin + d * cos], -1).flatten(-2)
    else:
        a, d = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * cos - d * sin, a * sin + d * cos], -1)
    return torch.cat([turned, rest], -1)


def _plain_append(s):
    c = s["case"]
    qh, kvh = c["query_heads"], c["kv_heads"]
    b, pos, live = _rows_of_sequences(s)
    q, k = s["qkv"][:, :qh].float(), s["qkv"][:, qh:qh + kvh].double()
    if c["norm"]:
        q, k = _norm(q, s["q_weight"]), _norm(k, s["k_weight"].double())
    q_out = torch.where(live[:, None, None], _turn(s, q, pos).half(), s["q_out"])
    n = s["total"] - c["pad_rows"]
    page = s["bt"].long()[b, pos.clamp(min=0) // c["page_size"]][:n]
    slot = (pos % c["page_size"])[:n]
    where = (page, slice(None), slot) if c["head_major"] else (page, slot)
    k, ks = _quantise(_turn(s, k, pos)[:n])
    v, vs = _quantise(s["qkv"][:n, qh + kvh:].double())
    s["k"][where], s["v"][where] = k, v
    s["ks"][page, :, slot], s["vs"][page, :, slot] = ks, vs
    return _cache_values(s, q_out)


def _values(s, codes, scale, page, slot):
    """Rows [..., kv_heads, head_dim] of the tokens at (page, slot), in 32 bits."""
    x = codes[page, :, slot] if s["case"]["head_major"] else codes[page, slot]
    e = scale[page, :, slot].float() - 127.0
    return x.view(torch.float8_e4m3fn).float() * torch.exp2(e)[..., None]


def _plain_read(s):
    c = s["case"]
    b, pos, live = _rows_of_sequences(s)
    pos = pos.clamp(min=0, max=s["max_ctx"] - 1)
    page, slot = s["bt"].long()[b, pos // c["page_size"]].clamp(min=0), pos % c["page_size"]
    live = live[:, None, None]
    return {"key": torch.where(live, _values(s, s["k"], s["ks"], page, slot).half(), s["k_out"]),
            "value": torch.where(live, _values(s, s["v"], s["vs"], page, slot).half(), s["v_out"])}


def _gather(s, codes, scale):
    """Every sequence's cached rows in token order: [batch][kv_heads][tokens][head_dim]."""
    c = s["case"]
    t = torch.arange(s["max_ctx"], device=DEV)
    page = s["bt"].long()[:, t // c["page_size"]].clamp(min=0)
    slot = (t % c["page_size"]).expand_as(page)
    return _values(s, codes, scale, page, slot).permute(0, 2, 1, 3)


def _plain_attention(s):
    c = s["case"]
    B, kvh, hd, T = c["batch"], c["kv_heads"], c["head_dim"], s["max_ctx"]
    g = c["query_heads"] // kvh
    ctx, out = s["ctx"].long(), s["out"]
    if T == 0:
        return torch.zeros_like(out)
    if c["op"] == "decode":
        n_rows, rows = 1, torch.arange(B, device=DEV)[:, None]
        pos = (ctx - 1)[:, None]
    else:
        n_rows, qs = s["max_new"], s["qs"].long()
        j = torch.arange(n_rows, device=DEV)
        rows = (qs[:-1, None] + j).clamp(max=s["total"] - 1)
        pos = (ctx - qs[1:] + qs[:-1])[:, None] + j
    q = s["q"][rows].float().view(B, n_rows, kvh, g, hd).permute(0, 2, 3, 1, 4)
    k = _gather(s, s["k"], s["ks"])
    x = q.reshape(B, kvh, g * n_rows, hd) @ k.transpose(-1, -2)
    x = x.view(B, kvh, g, n_rows, T) * s["scale"]
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    t = torch.arange(T, device=DEV)
    if c["alibi"]:
        away = (pos[..., None] - t).abs().float()
        x = x - s["slopes"].view(1, kvh, g, 1, 1) * away[:, None, None]
    last = pos
    if c["prefix"]:
        pre = s["prefix"].long()[:, None]
        last = torch.where(pos < pre, pre - 1, pos)
    last = torch.minimum(last, (ctx - 1)[:, None])
    lo = torch.zeros_like(pos)
    if c["window"]:
        lo = (pos - c["window"] + 1).clamp(min=0)
    if c["documents"]:
        lo = torch.maximum(lo, s["first"].long()[rows])
    seen = ((t <= last[..., None]) & (t >= lo[..., None]))[:, None, None]
    top = x.masked_fill(~seen, -math.inf).amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.where(seen, torch.exp(x - top), torch.zeros((), device=DEV))
    den = p.sum(-1, keepdim=True)
    v = _gather(s, s["v"], s["vs"])
    o = (p.view(B, kvh, g * n_rows, T) @ v).view(B, kvh, g, n_rows, hd)
    o = torch.where(den > 0, o / den, torch.zeros((), device=DEV))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n_rows, kvh * g, hd).to(out.dtype)
    if c["op"] == "decode":
        return o[:, 0]
    b, at, live = _rows_of_sequences(s)
    j = (at - (ctx - s["qs"][1:] + s["qs"][:-1])[b]).clamp(0, n_rows - 1)
    return torch.where(live[:, None, None], o[b, j], out)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return {"append": _plain_append, "read": _plain_read}.get(op, _plain_attention)(state)


# ------------------------------------------------------------------------------- 64 bits
def _code_table():
    """The 256 numbers of e4m3: sign, 4 bits of exponent (bias 7), 3 of mantissa; no infinities."""
    got = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        if e == 15 and m == 7:
            x = math.nan
        got.append(-x if code & 128 else x)
    return got


def _nearest(x):
    """Rows in 64 bits to (values that the codes stand for, scales), by search in the sorted
    positive codes."""
    grid = torch.tensor(_code_table()[:127], dtype=torch.float64, device=x.device)
    border = (grid[1:] + grid[:-1]) / 2
    top = x.abs().amax(-1)
    e = torch.full_like(top, -15.0)
    for k in range(-15, 8):
        e = torch.where(top > 448.0 * 2.0 ** k, k + 1.0, e)
    y = x.abs() * torch.exp2(-e)[..., None]
    y = torch.where((e == 8)[..., None], y.clamp(max=240.0), y)
    lower = torch.searchsorted(border, y.contiguous())             # a tie goes down ...
    upper = torch.searchsorted(border, y.contiguous(), right=True)  # ... or up:
    at = torch.where(lower % 2 == 0, lower, upper)                 # to the even code
    return torch.copysign(grid[at], x), torch.exp2(e)


def exact(case, seed):
    """Sequence by sequence from the definitions, in 64 bits."""
    s, c = prepare(case, seed), case
    ctx, new = _lengths(c)
    ps, kvh, qh, hd = c["page_size"], c["kv_heads"], c["query_heads"], c["head_dim"]
    start = np.concatenate([[0], np.cumsum(new)])
    bt = s["bt"].cpu().numpy()
    numbers = torch.tensor(_code_table(), dtype=torch.float64, device=DEV)

    def places(b, t):
        t = torch.as_tensor(np.asarray(t), device=DEV)
        return torch.from_numpy(bt[b].astype(np.int64)).to(DEV)[t // ps], t % ps

    def rows_of(codes, scale, b, t):
        page, slot = places(b, t)
        x = codes[page, :, slot] if c["head_major"] else codes[page, slot]
        return numbers[x.long()] * torch.exp2(scale[page, :, slot].double() - 127)[..., None]

    if c["op"] == "append":
        out = {"query": s["q_out"].double()}
        for x, codes, scale in (("key", s["k"], s["ks"]), ("value", s["v"], s["vs"])):
            out[x + "_cache"] = torch.empty(codes.shape, dtype=torch.float64, device=DEV)
            for to, part in zip(out[x + "_cache"].split(64), codes.split(64)):
                to.copy_(numbers[part.long()])
            out[x + "_scale"] = torch.exp2(scale.double() - 127)
        r = c["rotary"]
        first = torch.arange(0, r, 2, device=DEV) if c["interleaved"] else torch.arange(r // 2, device=DEV)
        second = first + (1 if c["interleaved"] else r // 2)
        for b in range(c["batch"]):
            if not new[b]:
                continue
            pos = np.arange(ctx[b] - new[b], ctx[b])
            rows = slice(int(start[b]), int(start[b + 1]))
            x = s["qkv"][rows].double()
            if c["norm"]:
                for heads, w in ((slice(0, qh), "q_weight"), (slice(qh, qh + kvh), "k_weight")):
                    size = torch.sqrt(x[:, heads].square().sum(-1, keepdim=True) / hd + EPS)
                    x[:, heads] = x[:, heads] / size * s[w].double()
            at = s["positions"][rows].long() if c["explicit"] else torch.as_tensor(pos, device=DEV)
            z = torch.complex(*(x[:, :qh + kvh][..., i] for i in (first, second)))
            z = z * torch.complex(*(s["table"][at, i].double() for i in (0, 1)))[:, None]
            x[:, :qh + kvh, first], x[:, :qh + kvh, second] = z.real, z.imag
            out["query"][rows] = x[:, :qh]
            page, slot = places(b, pos)
            where = (page, slice(None), slot) if c["head_major"] else (page, slot)
            for name, heads in (("key", slice(qh, qh + kvh)), ("value", slice(qh + kvh, None))):
                values, scale = _nearest(x[:, heads])
                out[name + "_cache"][where] = values
                out[name + "_scale"][page, :, slot] = scale
        return out

    if c["op"] == "read":
        got = {"key": s["k_out"].double(), "value": s["v_out"].double()}
        for b in range(c["batch"]):
            rows, pos = slice(int(start[b]), int(start[b + 1])), np.arange(ctx[b] - new[b], ctx[b])
            got["key"][rows] = rows_of(s["k"], s["ks"], b, pos)
            got["value"][rows] = rows_of(s["v"], s["vs"], b, pos)
        return got

    out = s["out"].double()
    seen = _visible(c)
    for b in range(c["batch"]):
        m, n = int(new[b]), int(ctx[b])
        rows = slice(b, b + 1) if c["op"] == "decode" else slice(int(start[b]), int(start[b + 1]))
        if m == 0:
            out[rows] = 0
            continue
        lo, hi = (torch.from_numpy(x.astype(np.int64)).to(DEV) for x in seen[b])
        t0, t1 = int(lo.min()), int(hi.max()) + 1
        t = torch.arange(t0, t1, device=DEV)
        pos = torch.arange(n - m, n, device=DEV)
        here = (t >= lo[:, None]) & (t <= hi[:, None])
        away = (pos[:, None] - t).abs().double()
        keys = rows_of(s["k"], s["ks"], b, np.arange(t0, t1))
        values = rows_of(s["v"], s["vs"], b, np.arange(t0, t1))
        for h in range(qh):
            kv = h // (qh // kvh)
            z = s["scale"] * (s["q"][rows, h].double() @ keys[:, kv].T)
            if c["softcap"]:
                z = c["softcap"] * torch.tanh(z / c["softcap"])
            if c["alibi"]:
                z = z - s["slopes"][h].double() * away
            weights = torch.softmax(z.masked_fill(~here, -math.inf), -1)
            out[rows, h] = weights @ values[:, kv]
    return out
