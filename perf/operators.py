"""The serving operators around the paged K/V cache: what is measured of them, and their plain
forms.

* ``append``  -- ``pa_append_rope``: the newest tokens' keys and values, taken from the fused
  projection's rows, are written into the paged caches with the position rotation applied to
  the keys on the way, and the rotated queries are packed for the attention call.
* ``decode``  -- ``pa_decode_scored``: one new token per sequence attends over the paged cache
  with scores capped by a tanh, a bias that grows with distance, a sliding window or a first
  visible token (a document's start).
* ``prefill`` -- ``pa_prefill_scored``: the same for several new tokens per sequence, with a
  prefix that sees itself in both directions.

``run`` computes the plain form in elementary torch operations in 32 bits, or, where ``own`` is
true, makes the calls a user makes. Sizes are those of the repository's workloads (tiny,
gqa4_mid, mha, long_gqa6, ragged and the multi-token ones) and of the range around them.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BASE = 10000.0  # of the rotation's frequencies


# ------------------------------------------------------------------------------- cases
def _case(name, op, **kw):
    c = dict(op=op, batch=2, query_heads=4, kv_heads=2, head_dim=64, page_size=16,
             head_major=False, ctx_lo=1, ctx_hi=64, new_lo=1, new_hi=1, pad_rows=0, mix=1)
    if op == "append":
        c.update(rotary=64, interleaved=False, explicit=False)
    else:
        c.update(softcap=0.0, window=0, alibi=False, documents=0, prefix=0, half_out=True)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # ---- append
        # one decode step of two short sequences: latency of the smallest call
        _case("append_step_tiny", "append", batch=2, ctx_lo=37, ctx_hi=100, mix=1),
        # one decode step of a full serving batch (the ragged workload's heads)
        _case("append_step_batch", "append", batch=256, query_heads=64, kv_heads=8, head_dim=128,
              page_size=32, ctx_lo=1, ctx_hi=1024, rotary=128, mix=2),
        # eight fresh 2048-token prompts written at once (prefill_gqa4's shape)
        _case("append_prompts", "append", batch=8, query_heads=32, kv_heads=8, head_dim=128,
              page_size=16, ctx_lo=2048, ctx_hi=2048, new_lo=2048, new_hi=2048, rotary=128, mix=3),
        # ragged chunks on cached prefixes: partial rotation of neighbouring pairs, positions
        # given by the caller, head-major pages, rows of a padded batch behind the last sequence
        _case("append_chunks_partial", "append", batch=13, query_heads=24, kv_heads=4,
              head_dim=256, page_size=64, head_major=True, ctx_lo=512, ctx_hi=4096, new_lo=1,
              new_hi=509, pad_rows=5, rotary=64, interleaved=True, explicit=True, mix=4),
        # ---- decode
        # two short sequences: latency
        _case("decode_tiny", "decode", batch=2, ctx_lo=37, ctx_hi=100, softcap=30.0, window=48,
              mix=5),
        # a mid-size batch (gqa4_mid) of a local layer: capped scores in a sliding window
        _case("decode_mid_window", "decode", batch=32, query_heads=32, kv_heads=8, head_dim=128,
              page_size=16, ctx_lo=512, ctx_hi=4096, softcap=30.0, window=1024, mix=6),
        # every head with keys of its own (mha), bias by distance, documents in one stream; the
        # output in 32 bits
        _case("decode_mha_distance", "decode", batch=64, query_heads=32, kv_heads=32,
              head_dim=128, page_size=16, ctx_lo=2048, ctx_hi=2048, alibi=True, documents=1500,
              half_out=False, mix=7),
        # four 100k-token contexts (long_gqa6) with capped scores: the longest reads
        _case("decode_long_cap", "decode", batch=4, query_heads=24, kv_heads=4, head_dim=256,
              page_size=64, ctx_lo=100000, ctx_hi=100000, softcap=50.0, mix=8),
        # ---- prefill
        # two short chunks: latency
        _case("prefill_tiny", "prefill", batch=2, ctx_lo=37, ctx_hi=100, new_lo=20, new_hi=37,
              softcap=30.0, mix=9),
        # eight 2048-token prompts (prefill_gqa4) through a local layer
        _case("prefill_window_cap", "prefill", batch=8, query_heads=32, kv_heads=8, head_dim=128,
              page_size=16, ctx_lo=2048, ctx_hi=2048, new_lo=2048, new_hi=2048, softcap=30.0,
              window=1024, mix=10),
        # chunked prefill (prefill_chunked) of packed documents with a bias by distance
        _case("prefill_documents_distance", "prefill", batch=16, query_heads=32, kv_heads=8,
              head_dim=128, page_size=16, ctx_lo=512, ctx_hi=4096, new_lo=512, new_hi=512,
              alibi=True, documents=700, mix=11),
        # two 4096-token prompts (prefill_gqa6_hd256) with a bidirectional prefix, capped
        _case("prefill_prefix_cap_hd256", "prefill", batch=2, query_heads=24, kv_heads=4,
              head_dim=256, page_size=64, ctx_lo=4096, ctx_hi=4096, new_lo=4096, new_hi=4096,
              softcap=50.0, prefix=1024, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {c["op"]: 0.0 for c in listed()}
    size = dict(most)
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most[c["op"]], max(w["bytes"], w["flops"] / 100))
        size[c["op"]] = max(size[c["op"]], _plain_size(c))
    while True:
        op = rng.choice(["append", "decode", "prefill"])
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
            c.update(rotary=rng.choice([0, 16, 32, 48, 64, hd, hd, hd]),
                     interleaved=rng.random() < 0.4, explicit=rng.random() < 0.3)
        else:
            c.update(softcap=rng.choice([0.0, 20.0, 30.0, 50.0]),
                     window=_log(rng, 1, 4096) if rng.random() < 0.4 else 0,
                     alibi=rng.random() < 0.35,
                     documents=_log(rng, 8, 4096) if rng.random() < 0.3 else 0,
                     half_out=op == "prefill" or rng.random() < 0.7)
            if op == "prefill" and rng.random() < 0.4:
                c["prefix"] = _log(rng, 1, 4096)
            if not (c["softcap"] or c["window"] or c["alibi"] or c["documents"]
                    or c.get("prefix", 0)):
                c["softcap"] = 30.0
        c = _case(None, op, **c)
        w = work(c)
        if max(w["bytes"], w["flops"] / 100) <= most[op] and _plain_size(c) <= size[op] \
                and w["bytes"] > 4096:
            return c


def _plain_size(c):
    """Values that the plain form holds at once: padded scores and gathered keys."""
    if c["op"] == "append":
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
    total, hd = int(new.sum()), c["head_dim"]
    if c["op"] == "append":
        rows = total * (c["query_heads"] + 2 * c["kv_heads"])
        turned = total * (c["query_heads"] + c["kv_heads"]) * c["rotary"]
        table = min(total, int(ctx.max())) * c["rotary"] * 4
        return {"bytes": 2.0 * rows * hd * 2 + table + 8.0 * total, "flops": 3.0 * turned}
    pairs = tokens = 0
    for lo, hi in _visible(c):
        if len(lo):
            pairs += int((hi - lo + 1).sum())
            tokens += int(hi.max() - lo.min() + 1)
    out_bytes = 2 if c["half_out"] else 4
    rows = total if c["op"] == "prefill" else c["batch"]
    return {"bytes": float(4.0 * tokens * c["kv_heads"] * hd
            + rows * c["query_heads"] * hd * (2.0 + out_bytes)
            + 4.0 * (-(-ctx // c["page_size"])).sum()),
            "flops": float(4.0 * hd * c["query_heads"] * pairs)}


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
    shape = (pages, kvh, ps, hd) if c["head_major"] else (pages, ps, kvh, hd)
    s = dict(case=dict(c), bt=ints(bt), ctx=ints(ctx), k=normal(*shape), v=normal(*shape),
             qs=ints(np.concatenate([[0], np.cumsum(new)])), total=total, maxp=maxp, pages=pages,
             scale=1.0 / math.sqrt(hd), max_ctx=int(ctx.max()), max_new=int(new.max()))
    if c["op"] == "append":
        # the fused projection's output: each token's query, key and value rows side by side
        s["qkv"] = normal(total, qh + 2 * kvh, hd)
        s["q_out"] = normal(total, qh, hd)
        half = c["rotary"] // 2
        rows = max(1, int(ctx.max()))
        turn = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * BASE ** (
            -torch.arange(half, device=DEV, dtype=torch.float64) / max(1, half))
        s["table"] = torch.stack([turn.cos(), turn.sin()], 1).float().contiguous()
        s["positions"] = None
        if c["explicit"]:
            s["positions"] = torch.randint(0, rows, (total,), generator=g, device=DEV,
                                           dtype=torch.int32)
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
    """What a serving program keeps beside its tensors: the problem, the rule and a workspace."""
    from paged_kv_cache_63_gb300 import lib

    c = s["case"]
    prob = lib.problem(c["batch"], c["query_heads"], c["kv_heads"], c["head_dim"],
                       c["page_size"], s["maxp"], s["pages"], int(c["head_major"]))
    if c["op"] == "append":
        rope = lib.rope(c["rotary"], "interleaved" if c["interleaved"] else "half", s["table"],
                        s["positions"])
        return dict(lib=lib, prob=prob, rope=rope)
    score = lib.score(softcap=c["softcap"], window=c["window"], slopes=s["slopes"],
                      first_tokens=s["first"], prefix_lengths=s["prefix"],
                      out="fp16" if c["half_out"] else "fp32")
    h = dict(lib=lib, prob=prob, score=score, ws=None, n=0)
    if c["op"] == "decode":
        h["n"] = lib.pa_workspace_size(prob)
        h["ws"] = torch.empty(max(h["n"], 256), dtype=torch.uint8, device=DEV)
    return h


def _run_own(s):
    c, h = s["case"], s["handle"]
    lib = h["lib"]
    if c["op"] == "append":
        qh, kvh = c["query_heads"], c["kv_heads"]
        qkv = s["qkv"]
        lib.pa_append_rope(h["prob"], h["rope"], qkv[:, :qh], qkv[:, qh:qh + kvh],
                           qkv[:, qh + kvh:], s["qs"], s["total"], s["bt"], s["ctx"], s["q_out"],
                           s["k"], s["v"])
        return {"query": s["q_out"], "key_cache": s["k"], "value_cache": s["v"]}
    if c["op"] == "decode":
        lib.pa_decode_scored(h["prob"], h["score"], s["q"], s["k"], s["v"], s["bt"], s["ctx"],
                             s["scale"], s["out"], workspace=h["ws"], workspace_bytes=h["n"])
    else:
        lib.pa_prefill_scored(h["prob"], h["score"], s["q"], s["qs"], s["total"], s["max_new"],
                              s["k"], s["v"], s["bt"], s["ctx"], s["scale"], s["out"])
    return s["out"]


# ------------------------------------------------------------------------------- plain forms
def _sequence_of_rows(s):
    """For each query row its sequence, its token's position, and whether it is a new token's."""
    row = torch.arange(s["total"], device=DEV)
    b = (torch.searchsorted(s["qs"].long(), row, right=True) - 1).clamp(0, s["case"]["batch"] - 1)
    qs, ctx = s["qs"].long(), s["ctx"].long()
    pos = ctx[b] - qs[b + 1] + row
    return b, pos, row < qs[-1]


def _plain_append(s):
    c = s["case"]
    qh, kvh, half = c["query_heads"], c["kv_heads"], c["rotary"] // 2
    b, pos, live = _sequence_of_rows(s)
    x = s["qkv"][:, :qh + kvh].float()
    if half:
        at = s["positions"].long() if c["explicit"] else pos.clamp(min=0, max=s["max_ctx"] - 1)
        cos, sin = (s["table"][at, i][:, None, :] for i in (0, 1))
        turned, rest = x[..., :2 * half], x[..., 2 * half:]
        if c["interleaved"]:
            a, d = turned[..., 0::2], turned[..., 1::2]
            turned = torch.stack([a * cos - d * sin, a * sin + d * cos], -1).flatten(-2)
        else:
            a, d = turned[..., :half], turned[..., half:]
            turned = torch.cat([a * cos - d * sin, a * sin + d * cos], -1)
        x = torch.cat([turned, rest], -1)
    x = x.half()
    q_out = torch.where(live[:, None, None], x[:, :qh], s["q_out"])
    n = s["total"] - c["pad_rows"]
    page = s["bt"].long()[b, pos.clamp(min=0) // c["page_size"]][:n]
    slot = (pos % c["page_size"])[:n]
    where = (page, slice(None), slot) if c["head_major"] else (page, slot)
    s["k"][where] = x[:n, qh:]
    s["v"][where] = s["qkv"][:n, qh + kvh:]
    return {"query": q_out, "key_cache": s["k"], "value_cache": s["v"]}


def _gather(s, cache):
    """Every sequence's cached rows in token order: [batch][kv_heads][tokens][head_dim], fp32."""
    c = s["case"]
    t = torch.arange(s["max_ctx"], device=DEV)
    page = s["bt"].long()[:, t // c["page_size"]].clamp(min=0)
    slot = (t % c["page_size"]).expand_as(page)
    x = cache[page, :, slot] if c["head_major"] else cache[page, slot]
    return x.permute(0, 2, 1, 3).float()


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
    k, v = _gather(s, s["k"]), _gather(s, s["v"])
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
    o = (p.view(B, kvh, g * n_rows, T) @ v).view(B, kvh, g, n_rows, hd)
    o = torch.where(den > 0, o / den, torch.zeros((), device=DEV))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n_rows, kvh * g, hd).to(out.dtype)
    if c["op"] == "decode":
        return o[:, 0]
    b, at, live = _sequence_of_rows(s)
    j = (at - (ctx - s["qs"][1:] + s["qs"][:-1])[b]).clamp(0, n_rows - 1)
    return torch.where(live[:, None, None], o[b, j], out)


def run(state):
    if own:
        return _run_own(state)
    return _plain_append(state) if state["case"]["op"] == "append" else _plain_attention(state)


# ------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """Sequence by sequence from the definitions, in 64 bits."""
    s, c = prepare(case, seed), case
    ctx, new = _lengths(c)
    ps, kvh, qh, hd = c["page_size"], c["kv_heads"], c["query_heads"], c["head_dim"]
    start = np.concatenate([[0], np.cumsum(new)])
    bt = s["bt"].cpu().numpy()

    def places(b, t):
        t = torch.as_tensor(np.asarray(t), device=DEV)
        page = torch.from_numpy(bt[b].astype(np.int64)).to(DEV)[t // ps]
        return (page, slice(None), t % ps) if c["head_major"] else (page, t % ps)

    if c["op"] == "append":
        q_out, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
        r = c["rotary"]
        first = torch.arange(0, r, 2, device=DEV) if c["interleaved"] else torch.arange(r // 2, device=DEV)
        second = first + (1 if c["interleaved"] else r // 2)
        for b in range(c["batch"]):
            if not new[b]:
                continue
            pos = np.arange(ctx[b] - new[b], ctx[b])
            rows = slice(int(start[b]), int(start[b + 1]))
            x = s["qkv"][rows].double()
            at = s["positions"][rows].long() if c["explicit"] else torch.as_tensor(pos, device=DEV)
            z = torch.complex(*(x[:, :qh + kvh][..., i] for i in (first, second)))
            z = z * torch.complex(*(s["table"][at, i].double() for i in (0, 1)))[:, None]
            x[:, :qh + kvh, first], x[:, :qh + kvh, second] = z.real, z.imag
            q_out[rows] = x[:, :qh]
            k[places(b, pos)] = x[:, qh:qh + kvh]
            v[places(b, pos)] = x[:, qh + kvh:]
        return {"query": q_out, "key_cache": k, "value_cache": v}

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
        keys, values = (s[x][places(b, np.arange(t0, t1))] for x in ("k", "v"))
        for h in range(qh):
            kv = h // (qh // kvh)
            z = s["scale"] * (s["q"][rows, h].double() @ keys[:, kv].double().T)
            if c["softcap"]:
                z = c["softcap"] * torch.tanh(z / c["softcap"])
            if c["alibi"]:
                z = z - s["slopes"][h].double() * away
            weights = torch.softmax(z.masked_fill(~here, -math.inf), -1)
            out[rows, h] = weights @ values[:, kv].double()
    return out
