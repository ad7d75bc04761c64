"""Measured cases of the 4-bit KV cache operators: append, attention (with and without
per-position attention weights) and eviction.

The cache holds each K and V row in blocks of 32 consecutive head dimensions, one fp16
scale d and 32 4-bit codes u per block, value = d * (u - 8), with d = fp16(max|x| / 7) and
u = clamp(rint(x / d), -8, 7) + 8 (all codes 8 where d is 0).

``run`` with ``own`` false computes each operator in elementary torch operations; with
``own`` true it makes the library's calls.  Sequence lengths are part of a case (spread
over its range by slot), values are made from the seed.
"""
from __future__ import annotations

import random

import numpy as np
import torch

own = False

BLOCK = 32
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def _case(op, dtype, slots, heads, kv_heads, head_dim, tokens, lo, hi, budget=0, sink=0, recent=0):
    return {"op": op, "dtype": dtype, "slots": slots, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "tokens": tokens, "lo": lo, "hi": hi, "budget": budget,
            "sink": sink, "recent": recent}


def listed():
    def named(name, c):
        return dict(c, name=name)

    return [
        # one decode step's new K / V rows of the batched Llama-8B workload, 64 slots at 512..4096
        named("append_step_b64", _case("append", "bf16", 64, 32, 8, 128, 1, 512, 4096)),
        # four ragged prompts in one padded batch, from an fp32 projection
        named("append_ragged_fp32", _case("append", "fp32", 4, 32, 8, 128, 1031, 0, 0)),
        # one long prompt of an MHA model (Llama-7B heads) moved into the 4-bit cache
        named("append_prompt_8k", _case("append", "bf16", 1, 32, 32, 128, 8191, 0, 0)),
        # the tiny model's heads on a short context: latency only
        named("attn_tiny", _case("attention", "fp32", 1, 8, 4, 32, 1, 99, 99)),
        # single-sequence decode at Llama-7B heads and its benchmark context
        named("attn_b1_mha_2k", _case("attention", "fp32", 1, 32, 32, 128, 1, 2049, 2049)),
        # the batched Llama-8B workload: 64 ragged slots
        named("attn_b64_gqa", _case("attention", "fp32", 64, 32, 8, 128, 1, 512, 4096)),
        # two very long contexts: the cache split over the whole GPU
        named("attn_long_128k", _case("attention", "bf16", 2, 32, 8, 128, 1, 100003, 131071)),
        # verification of five drafted tokens per slot, short and long slots, head_dim 64
        named("attn_draft5_hd64", _case("attention", "bf16", 16, 16, 2, 64, 5, 3, 3001)),
        # decode attention that also leaves every position's weight, for the eviction
        named("track_b8_gqa", _case("track", "fp32", 8, 32, 8, 128, 1, 512, 4096)),
        # a prompt scored by its last 16 queries, MHA
        named("track_window16", _case("track", "bf16", 1, 32, 32, 128, 16, 6007, 6007)),
        # slots around a budget of 1024: some one entry over it, some below
        named("evict_budget_1k", _case("evict", "bf16", 64, 32, 8, 128, 1, 900, 1100, 1024, 4, 256)),
        # long prompts cut to a quarter before decoding
        named("evict_32k_to_8k", _case("evict", "bf16", 4, 32, 8, 128, 1, 30011, 32767, 8192, 4, 64)),
    ]


def _logint(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "track", "evict"])
    dtype = rng.choice(["fp32", "bf16"])
    head_dim = rng.choice([32, 64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 32])
    group = rng.choice([1, 2, 3, 4, 7, 8]) if kv_heads < 32 else 1
    slots = _logint(rng, 1, 64)
    # positions over all slots and heads stay below the largest listed case
    most = (1 << 21) * 128 // head_dim // kv_heads // slots
    if op == "append":
        tokens = _logint(rng, 1, max(2, min(8191, most // 8)))
        hi = 0 if tokens > 64 or rng.random() < 0.3 else _logint(rng, 1, max(2, min(8192, most // 4)))
        return _case(op, dtype, slots, kv_heads * group, kv_heads, head_dim, tokens, min(hi, rng.randint(0, 512)), hi)
    if op == "evict":
        hi = _logint(rng, 64, max(65, min(32767, most // 2)))
        lo = max(1, int(hi * rng.uniform(0.3, 1.0)))
        budget = max(33, int(hi * rng.choice([0.25, 0.5, 0.9, 0.99]) * rng.uniform(0.9, 1.0)))
        sink = rng.choice([0, 4, 7])
        return _case(op, dtype, slots, kv_heads * group, kv_heads, head_dim, 1, lo, hi, budget, sink,
                     rng.randint(0, budget - sink))
    tokens = rng.choice([1, 1, 1, 2, 3, 5, 8])
    tokens = max(1, min(tokens, 64 // group))
    hi = _logint(rng, 2, max(3, min(131071, most // (1 + tokens * group // 8))))
    return _case(op, dtype, slots, kv_heads * group, kv_heads, head_dim, tokens, max(1, int(hi * rng.random())), hi)


def _spread(lo, hi, n, salt):
    """n lengths in [lo, hi], the same for a case each time, the range's ends among them."""
    r = random.Random(1000003 * lo + 1009 * hi + 7 * n + salt)
    out = [hi if i == n // 2 else lo if i == 0 and n > 1 else r.randint(lo, hi) for i in range(n)]
    return out


def _lengths(c):
    return _spread(c["lo"], c["hi"], c["slots"], 1)


def _new(c):
    """Appended tokens per slot: all in a decode step, ragged prompts otherwise."""
    T = c["tokens"]
    return [T] * c["slots"] if T <= 8 else _spread((T + 1) // 2, T, c["slots"], 2)


def _cap(c):
    n = c["hi"] + (c["tokens"] if c["op"] == "append" else 0)
    return -(-max(n, 1) // 32) * 32


# ----------------------------------------------------------------- inputs
def _randn(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _inputs(c, seed):
    """Rows as a model makes them: keys with a few strong channels, values whose size differs
    by position, queries that give some positions most of the weight."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, H, Hkv, hd, T = c["slots"], c["heads"], c["kv_heads"], c["head_dim"], c["tokens"]
    dt = DTYPES[c["dtype"]]
    d = {"lens": torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")}
    chan = 1.0 + 3.0 * (torch.rand((1, 1, Hkv, hd), generator=gen, device="cuda") < 0.05).float()

    def rows(n, dtype):
        k = torch.randn((B, n, Hkv, hd), generator=gen, device="cuda").mul_(chan).to(dtype)
        v = torch.randn((B, n, Hkv, hd), generator=gen, device="cuda")
        v.mul_(0.25 + torch.rand((B, n, 1, 1), generator=gen, device="cuda"))
        return k, v.to(dtype)

    # what the cache holds before the call
    d["k0"], d["v0"] = rows(_cap(c), torch.bfloat16) if c["hi"] else (None, None)
    if c["op"] == "append":
        d["k"], d["v"] = rows(T, dt)
        d["n_new"] = torch.tensor(_new(c), dtype=torch.int32, device="cuda")
    elif c["op"] == "evict":
        # sums of softmax weights over many steps: a few heavy entries, many light, some exactly alike
        w = torch.rand((B, Hkv, _cap(c)), generator=gen, device="cuda").clamp_(min=1e-6).reciprocal_()
        d["weights"] = torch.where(w < 1.05, torch.full_like(w, 1.0), w)
        inside = torch.arange(_cap(c), device="cuda") < d["lens"][:, None, None]
        d["weights"] = torch.where(inside, d["weights"], torch.zeros_like(w))
    else:
        d["q"] = _randn((B, T, H, hd), gen, torch.float32).mul_(1.5).to(dt)
    return d


# ------------------------------------------------------------- plain form
def _quantise(x):
    """Codes (uint8) and fp16 scales of rows x [..., head_dim]."""
    x = x.float()
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // BLOCK, BLOCK))
    top = b.abs().amax(-1)
    d = (top / torch.full_like(top, 7.0)).to(torch.float16)   # a true division, not a product with 1/7
    s = d.float()[..., None]
    u = torch.where(s > 0, (b / s).round().clamp(-8, 7), torch.zeros_like(b)) + 8
    return u.to(torch.uint8).reshape(x.shape), d


def _values(u, d):
    b = u.float().reshape(u.shape[:-1] + (d.shape[-1], BLOCK)) - 8.0
    return (b * d.float()[..., None]).reshape(u.shape)


def _plain_cache(c, d):
    B, Hkv, hd, cap = c["slots"], c["kv_heads"], c["head_dim"], _cap(c)
    s = {}
    for n, x in (("k", d["k0"]), ("v", d["v0"])):
        if x is None:
            u = torch.zeros((B, Hkv, cap, hd), dtype=torch.uint8, device="cuda")
            sc = torch.zeros((B, Hkv, cap, hd // BLOCK), dtype=torch.float16, device="cuda")
        else:
            u, sc = _quantise(x)
            u, sc = u.transpose(1, 2).contiguous(), sc.transpose(1, 2).contiguous()
        s["u" + n], s["d" + n] = u, sc
    return s


def _plain_append(s):
    T = s["k"].shape[1]
    B, Hkv, cap, hd = s["uk"].shape
    t = torch.arange(T, device="cuda")
    pos = s["lens"].long()[:, None] + t
    ok = t < s["n_new"][:, None]
    b, tt = torch.nonzero(ok, as_tuple=True)
    p = pos[b, tt]
    out = []
    for n in "kv":
        u, d = _quantise(s[n])
        s["u" + n][b, :, p] = u[b, tt]
        s["d" + n][b, :, p] = d[b, tt]
        y = torch.zeros((B, T, Hkv, hd), dtype=torch.float32, device="cuda")
        y[b, tt] = _values(s["u" + n][b, :, p], s["d" + n][b, :, p])
        out.append(y)
    return {"k": out[0], "v": out[1], "lens": s["lens"] + s["n_new"]}


def _plain_attention(s, track):
    q = s["q"].float()
    B, T, H, hd = q.shape
    Hkv, cap = s["uk"].shape[1:3]
    G = H // Hkv
    k, v = _values(s["uk"], s["dk"]), _values(s["uv"], s["dv"])
    rows = q.reshape(B, T, Hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, hd)
    x = torch.matmul(rows, k.transpose(2, 3)) * (hd ** -0.5)
    limit = s["lens"][:, None] - T + 1 + torch.arange(T, device="cuda")
    limit = limit.repeat_interleave(G, dim=1)[:, None, :, None]
    seen = torch.arange(cap, device="cuda") < limit
    x = torch.where(seen, x, torch.full_like(x, float("-inf")))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-38)
    o = torch.matmul(p, v)
    o = o.reshape(B, Hkv, T, G, hd).permute(0, 2, 1, 3, 4).reshape(B, T, H, hd).to(s["q"].dtype)
    return {"out": o, "weights": p.sum(2)} if track else {"out": o}


def _plain_evict(s):
    c, w = s["case"], s["weights"]
    B, Hkv, cap = w.shape
    m = c["budget"]
    n = s["lens"].long()[:, None, None]
    i = torch.arange(cap, device="cuda").expand(B, Hkv, cap)
    inside = i < n
    safe = inside & ((i < c["sink"]) | (i >= n - c["recent"]))
    key = torch.where(safe, torch.full_like(w, float("inf")), w)
    key = torch.where(inside, key, torch.full_like(w, float("-inf")))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    keep = torch.zeros((B, Hkv, cap), dtype=torch.bool, device="cuda")
    keep.scatter_(2, order[..., :min(m, cap)], True)
    keep = torch.where(n <= m, inside, keep & inside)
    front = i < m
    hole, mover = inside & front & ~keep, keep & ~front
    # the r-th hole takes the r-th kept entry behind the budget
    movers = torch.sort(torch.where(mover, i, torch.full_like(i, cap)), dim=-1).values
    rank = torch.cumsum(hole.long(), -1) - 1
    src = torch.where(hole, torch.gather(movers, 2, rank.clamp(min=0)), i)[..., :m].clamp(max=cap - 1)
    lens = torch.minimum(s["lens"], torch.full_like(s["lens"], m))
    live = torch.arange(src.shape[-1], device="cuda") < lens[:, None, None]
    out = {"lens": lens, "ids": torch.where(live, src, torch.zeros_like(src)).to(torch.int32),
           "weights": torch.where(live, torch.gather(w, 2, src), torch.zeros((), device="cuda"))}
    for name in "kv":
        u = torch.gather(s["u" + name], 2, src[..., None].expand(-1, -1, -1, s["u" + name].shape[-1]))
        d = torch.gather(s["d" + name], 2, src[..., None].expand(-1, -1, -1, s["d" + name].shape[-1]))
        y = torch.where(live[..., None], _values(u, d), torch.zeros((), device="cuda"))
        out[name] = y.transpose(1, 2).to(torch.bfloat16).contiguous()
    return out


# ------------------------------------------------------------- measured calls
def prepare(case, seed):
    d = _inputs(case, seed)
    s = {"case": case, **{n: d.get(n) for n in ("k", "v", "n_new", "q", "lens", "weights")}}
    B, Hkv, hd, T, op = case["slots"], case["kv_heads"], case["head_dim"], case["tokens"], case["op"]
    if op == "evict":
        s["yk"] = torch.empty((B, min(case["budget"], _cap(case)), Hkv, hd), dtype=torch.bfloat16, device="cuda")
        s["yv"] = torch.empty_like(s["yk"])
    elif op == "append":
        s["yk"] = torch.empty((B, T, Hkv, hd), dtype=torch.float32, device="cuda")
        s["yv"] = torch.empty_like(s["yk"])
    else:
        s["out"] = torch.empty_like(s["q"])
    if own:
        import transformer_decode_step_gb300 as pnb

        def cache(cap, track=0):
            x = pnb.Kv4Cache(n_layer=1, n_slot=B, n_head=case["heads"], n_kv_head=Hkv, head_dim=hd,
                             cap=cap, track=track)
            x.reset()
            return x

        s["cache"] = cache(_cap(case), T if op == "track" else 0)
        if d["k0"] is not None:
            s["cache"].append(0, d["k0"], d["v0"], n_new=s["lens"])
        if op == "evict":
            s["cache"].weights(0).copy_(s["weights"])
            s["kept"] = cache(-(-case["budget"] // 32) * 32)
            s["kept"].weights(0).zero_()
            s["kept"].ids(0).zero_()
        elif op == "track":
            s["cache"].weights(0).zero_()
    else:
        s.update(_plain_cache(case, d))
    return s


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "append":
            return _plain_append(s)
        if op == "evict":
            return _plain_evict(s)
        return _plain_attention(s, op == "track")
    cache = s["cache"]
    if op == "append":
        cache.append(0, s["k"], s["v"], n_new=s["n_new"], start=s["lens"])
        cache.read(0, s["yk"], s["yv"], first=s["lens"])
        return {"k": s["yk"], "v": s["yv"], "lens": cache.lengths(0)}
    if op == "evict":
        kept = s["kept"]
        cache.evict(0, c["budget"], n_sink=c["sink"], n_recent=c["recent"], dst=kept)
        kept.read(0, s["yk"], s["yv"])
        m = s["yk"].shape[1]
        return {"lens": kept.lengths(0), "ids": kept.ids(0)[..., :m], "weights": kept.weights(0)[..., :m],
                "k": s["yk"], "v": s["yv"]}
    if op == "track":
        cache.attention(0, s["q"], s["out"], decay=0.0)
        return {"out": s["out"], "weights": cache.weights(0)}
    cache.attention(0, s["q"], s["out"])
    return {"out": s["out"]}


def work(case):
    c = case
    H, Hkv, hd, T, op = c["heads"], c["kv_heads"], c["head_dim"], c["tokens"], c["op"]
    es = 4 if c["dtype"] == "fp32" else 2
    entry = 2 * (hd // 2 + hd // 16)              # one position's K and V of one head in the cache
    if op == "append":
        n = sum(_new(c)) * Hkv
        # rows in, codes out, every row of the read-back out
        return {"bytes": n * (2 * hd * es + entry) + 8 * c["slots"] * T * Hkv * hd, "flops": 6 * n * 2 * hd}
    lens = _lengths(c)
    if op == "evict":
        kept = sum(min(n, c["budget"]) for n in lens) * Hkv
        rows = c["slots"] * Hkv * min(c["budget"], _cap(c))
        return {"bytes": 8 * sum(lens) * Hkv + kept * (2 * entry + 8) + rows * 4 * hd, "flops": 8 * sum(lens) * Hkv}
    nbytes = sum(lens) * Hkv * entry + 2 * c["slots"] * T * H * hd * es
    if op == "track":
        nbytes += 4 * sum(lens) * Hkv
    return {"bytes": nbytes, "flops": 4 * T * H * hd * sum(lens)}


# ---------------------------------------------------------- in 64 bits
def _held64(x):
    """The values the cache stands for, rows x [..., head_dim], in 64 bits."""
    y = x.double().unflatten(-1, (-1, BLOCK))
    top = torch.maximum(y.max(-1).values, -y.min(-1).values)
    d = torch.from_numpy((top / 7).cpu().numpy().astype(np.float16).astype(np.float64)).to(x.device)
    d = d.unsqueeze(-1)
    code = torch.round(y / torch.where(d == 0, torch.ones_like(d), d))
    return (torch.minimum(torch.maximum(code, torch.full_like(code, -8.0)), torch.full_like(code, 7.0)) * d).flatten(-2)


def exact(case, seed):
    c, d = case, _inputs(case, seed)
    B, H, Hkv, hd, T = c["slots"], c["heads"], c["kv_heads"], c["head_dim"], c["tokens"]
    if c["op"] == "append":
        r = {}
        for n in "kv":
            y = _held64(d[n])
            for b, m in enumerate(_new(c)):
                y[b, m:] = 0
            r[n] = y
        return {"k": r["k"], "v": r["v"], "lens": None}
    if c["op"] == "evict":
        m = min(c["budget"], _cap(c))
        w = d["weights"].cpu().numpy()
        src = np.full((B, Hkv, m), -1, dtype=np.int64)
        for b, n in enumerate(_lengths(c)):
            for h in range(Hkv):
                if n <= m:
                    src[b, h, :n] = np.arange(n)
                    continue
                at = np.arange(n)
                fixed = (at < c["sink"]) | (at >= n - c["recent"])
                loose = at[~fixed]
                best = loose[np.lexsort((loose, -w[b, h, loose].astype(np.float64)))]
                kept = np.zeros(n, dtype=bool)
                kept[fixed] = True
                kept[best[: m - int(fixed.sum())]] = True
                row = np.where(kept[:m], np.arange(m), -1)
                row[row < 0] = np.flatnonzero(kept[m:]) + m
                src[b, h] = row
        live = src >= 0
        out = {"lens": None, "ids": None,
               "weights": torch.from_numpy(np.where(live, np.take_along_axis(w, src.clip(0), 2), 0).astype(np.float64))}
        at = torch.from_numpy(src.clip(0)).to("cuda").transpose(1, 2)[..., None].expand(-1, -1, -1, hd)
        for n in "kv":
            y = torch.gather(_held64(d[n + "0"]), 1, at)
            out[n] = y * torch.from_numpy(live).to("cuda").transpose(1, 2)[..., None]
        return out
    k, v = _held64(d["k0"]), _held64(d["v0"])
    q = d["q"].double()
    G = H // Hkv
    out = torch.zeros((B, T, H, hd), dtype=torch.float64, device="cuda")
    weights = torch.zeros((B, Hkv, _cap(c)), dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(c)):
        for t in range(T):
            m = n - T + 1 + t
            if m <= 0:
                continue
            for g in range(G):  # query heads g, G + g, 2G + g, ... of all KV heads at once
                z = torch.einsum("hd,nhd->hn", q[b, t, g::G], k[b, :m]) / hd ** 0.5
                p = torch.softmax(z, -1)
                out[b, t, g::G] = torch.einsum("hn,nhd->hd", p, v[b, :m])
                weights[b, :, :m] += p
    return {"out": out, "weights": weights} if c["op"] == "track" else {"out": out}
