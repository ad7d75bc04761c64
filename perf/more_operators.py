"""Measured cases of the paged KV cache operators: append with the position rotation, attention
of packed prompts, and decode attention of sequences that share a prefix.

A pool holds pages of ``page`` entries, [n_page][2 (K, V)][kv_heads][page][head_dim] in bf16.
Entry i of a sequence lies in row i % page of the page that its page table names at i // page.
``len`` counts a sequence's entries, this call's tokens included; token t of the n that a
sequence has in a call is its entry len - n + t.

``run`` with ``own`` false computes each operator in elementary torch operations; with ``own``
true it makes the library's calls.  Lengths are part of a case (spread over its ranges by
sequence); values and the order of the pages are made from the seed.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def _case(op, dtype, heads, kv_heads, head_dim, page, seqs, new, old, window=0, neox=False, axes=1,
          theta=10000.0, groups=0, prefix=(0, 0)):
    """new, old, prefix: (least, most) tokens of a sequence in the call, entries before them
    (behind the shared prefix), entries of a group's prefix."""
    return {"op": op, "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "seqs": seqs, "new_lo": new[0], "new_hi": new[1], "old_lo": old[0], "old_hi": old[1],
            "window": window, "neox": neox, "axes": axes, "theta": theta, "groups": groups,
            "prefix_lo": prefix[0], "prefix_hi": prefix[1]}


def listed():
    def named(name, c):
        return dict(c, name=name)

    return [
        # one decode step's rows of the batched Llama-8B workload: 64 slots at 512..4096
        named("append_step_b64", _case("append", "bf16", 32, 8, 128, 64, 64, (1, 1), (512, 4096))),
        # five ragged prompts and prompt chunks from an fp32 projection, small pages
        named("append_ragged_fp32", _case("append", "fp32", 32, 8, 128, 16, 5, (1, 1031), (0, 200))),
        # one long prompt of an MHA model (Llama-7B heads), the half-split rotation
        named("append_prompt_8k", _case("append", "bf16", 32, 32, 128, 128, 1, (8191, 8191), (0, 0), neox=True)),
        # two videos between text: positions over time, height and width
        named("append_video_axes", _case("append", "bf16", 16, 2, 128, 32, 2, (2500, 2731), (0, 77), neox=True,
                                         axes=3, theta=1000000.0)),
        # a short chat turn on few heads: latency only
        named("prompt_tiny", _case("prompt", "fp32", 8, 4, 64, 16, 1, (13, 13), (0, 0))),
        # sixteen users' prompts of one scheduler step, packed
        named("prompt_packed16", _case("prompt", "bf16", 32, 8, 128, 64, 16, (33, 2048), (0, 0))),
        # one long document
        named("prompt_16k", _case("prompt", "bf16", 32, 8, 128, 128, 1, (16383, 16383), (0, 0))),
        # the next 512 tokens of a long context (chunked prefill): few rows, a long axis
        named("prompt_chunk_60k", _case("prompt", "bf16", 32, 8, 128, 64, 1, (512, 512), (60001, 60001))),
        # two prompts under the Mistral window, queries as the projection leaves them in fp32
        named("prompt_window_fp32", _case("prompt", "fp32", 32, 8, 128, 64, 2, (5000, 8191), (0, 0), window=4096)),
        # a few requests behind a short system prompt: latency
        named("shared_tiny", _case("shared", "bf16", 16, 2, 64, 16, 4, (1, 1), (1, 40), groups=1, prefix=(512, 512))),
        # 64 requests behind one long system prompt, the step's own fp32 queries
        named("shared_b64", _case("shared", "fp32", 32, 8, 128, 64, 64, (1, 1), (0, 1024), groups=1,
                                  prefix=(8192, 8192))),
        # four documents with eight questions each, five drafted tokens to verify
        named("shared_draft5", _case("shared", "bf16", 32, 8, 128, 32, 32, (5, 5), (3, 700), groups=4,
                                     prefix=(2048, 30016))),
    ]


def _logint(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["append", "prompt", "prompt", "shared"])
    dtype = rng.choice(["fp32", "bf16", "bf16"])
    head_dim = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 32])
    heads = kv_heads * (rng.choice([1, 2, 3, 4, 7, 8]) if kv_heads < 32 else 1)
    window = 0 if rng.random() < 0.7 else _logint(rng, 16, 4096)
    if op == "append":
        new = _logint(rng, 1, 8191)
        seqs = _logint(rng, 1, max(1, min(64, 262144 // (new * heads))))
        old = rng.choice([0, _logint(rng, 1, min(4096, 262144 // seqs // kv_heads))])
        axes = rng.choice([1, 1, 3])
        return _case(op, dtype, heads, kv_heads, head_dim, page, seqs, (rng.randint(1, new), new),
                     (rng.randint(0, old), old), neox=rng.random() < 0.5, axes=axes,
                     theta=rng.choice([10000.0, 500000.0, 1000000.0]))
    if op == "prompt":
        if rng.random() < 0.3:      # a chunk on a long context
            seqs, new, old = _logint(rng, 1, 4), _logint(rng, 2, 600), _logint(rng, 1000, 60000)
        else:
            new = _logint(rng, 2, 16383)
            seqs, old = _logint(rng, 1, max(1, min(32, 16384 // new))), 0
        while seqs * heads * new * (new + old) > 1 << 32 or seqs * (new + old) * kv_heads > 1 << 20:
            new, old = -(-new * 2 // 3), old * 2 // 3
        return _case(op, dtype, heads, kv_heads, head_dim, page, seqs, (rng.randint(1, new), new),
                     (rng.randint(old // 2, old), old), window)
    groups = rng.choice([1, 1, 2, 4])
    seqs = groups * _logint(rng, 2, 64 // groups)
    T = rng.choice([1, 1, 1, 2, 5])
    old = _logint(rng, 1, 2048)
    prefix = _logint(rng, page, 32768)
    while seqs * (prefix + old) * kv_heads > 1 << 22:
        prefix, old = prefix * 2 // 3, -(-old * 2 // 3)
    prefix = -(-prefix // page) * page
    return _case(op, dtype, heads, kv_heads, head_dim, page, seqs, (T, T), (rng.randint(0, old), old), window,
                 groups=groups, prefix=(max(page, int(prefix * rng.random()) // page * page), prefix))


def _spread(lo, hi, n, salt):
    """n numbers in [lo, hi], the same for a case each time, the range's ends among them."""
    r = random.Random(1000003 * lo + 1009 * hi + 7 * n + salt)
    return [hi if i == n // 2 else lo if i == 0 and n > 1 else r.randint(lo, hi) for i in range(n)]


def _new(c):
    return _spread(c["new_lo"], c["new_hi"], c["seqs"], 1)


def _prefix(c):
    """The shared entries of every group, whole pages."""
    return [p // c["page"] * c["page"] for p in _spread(c["prefix_lo"], c["prefix_hi"], c["groups"], 3)]


def _lens(c):
    lens = [n + o for n, o in zip(_new(c), _spread(c["old_lo"], c["old_hi"], c["seqs"], 2))]
    if c["groups"]:
        each = c["seqs"] // c["groups"]
        lens = [n + _prefix(c)[b // each] for b, n in enumerate(lens)]
    return lens


def _sections(c):
    """Pairs of a head that turn by each position axis."""
    half = c["head_dim"] // 2
    return [half // 4, half * 3 // 8, half * 3 // 8] if c["axes"] == 3 else [half]


# ----------------------------------------------------------------- inputs
def _inputs(c, seed):
    """Rows as a model makes them: keys with a few strong channels, values whose size differs
    by position, queries that give some positions most of the weight."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    H, Hkv, hd, page = c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    dt = DTYPES[c["dtype"]]
    new, lens = _new(c), _lens(c)
    B, n_tok = c["seqs"], sum(new)
    max_page = max(-(-n // page) for n in lens)
    # page tables: a random order of the pool's pages, a group's first ones in common
    need = [-(-n // page) for n in lens]
    shared = [0] * B
    if c["groups"]:
        each = B // c["groups"]
        shared = [_prefix(c)[b // each] // page for b in range(B)]
    table = torch.zeros((B, max_page), dtype=torch.int64)
    n_page = 0
    for b in range(B):
        first = 0
        if c["groups"] and b % each:
            first = shared[b]
            table[b, :first] = table[b - b % each, :first]
        table[b, first:need[b]] = torch.arange(n_page, n_page + need[b] - first)
        n_page += need[b] - first
    n_page += 2
    order = torch.randperm(n_page, generator=gen, device="cuda")
    d = {"pages": order[table.cuda()].to(torch.int32), "n_page": n_page}
    d["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ends = [0]
    for n in new:
        ends.append(ends[-1] + n)
    d["start"] = torch.tensor(ends, dtype=torch.int32, device="cuda") if len(set(new)) > 1 else None
    chan = 1.0 + 3.0 * (torch.rand((Hkv, 1, hd), generator=gen, device="cuda") < 0.05).float()
    pool = torch.empty((n_page, 2, Hkv, page, hd), dtype=torch.bfloat16, device="cuda")
    for i in range(0, n_page, 1024):
        part = torch.randn((min(1024, n_page - i), 2, Hkv, page, hd), generator=gen, device="cuda")
        part[:, 0].mul_(chan)
        part[:, 1].mul_(0.25 + torch.rand((part.shape[0], 1, page, 1), generator=gen, device="cuda"))
        pool[i:i + 1024] = part
    d["pool"] = pool
    d["q"] = torch.randn((n_tok, H, hd), generator=gen, device="cuda").mul_(1.5).to(dt)
    if c["op"] == "append":
        d["k"] = torch.randn((n_tok, Hkv, hd), generator=gen, device="cuda").mul_(chan[:, 0]).to(dt)
        d["v"] = torch.randn((n_tok, Hkv, hd), generator=gen, device="cuda").to(dt)
        if c["axes"] == 3:
            # frames of a picture grid: time, row and column
            t = torch.arange(n_tok, device="cuda")
            off = torch.randint(0, 500, (1,), generator=gen, device="cuda")
            d["pos"] = torch.stack([off + t // 420, off + t // 21 % 20, off + t % 21]).to(torch.int32).contiguous()
    if c["groups"]:
        d["group_start"] = torch.arange(0, B + 1, each, dtype=torch.int32, device="cuda")
        d["prefix"] = torch.tensor(_prefix(c), dtype=torch.int32, device="cuda")
    return d


# ------------------------------------------------------------- plain form
def _tokens(s):
    """Sequence and entry of every packed token."""
    lens = s["lens"].long()
    B, n_tok = lens.numel(), s["q"].shape[0]
    start = s["start"]
    start = torch.arange(B + 1, device="cuda") * (n_tok // B) if start is None else start.long()
    t = torch.arange(n_tok, device="cuda")
    b = torch.searchsorted(start[1:], t, right=True)
    return b, lens[b] - start[b + 1] + t


def _rotate(x, pos, c):
    """Rows x [n_tok][heads][head_dim]; pos [axes][n_tok]."""
    hd = c["head_dim"]
    half = hd // 2
    p = torch.arange(half, device="cuda", dtype=torch.float64)
    freq = torch.exp(p * (-2.0 * math.log(c["theta"]) / hd))
    if c["axes"] == 3:
        s = _sections(c)
        at = pos.double()[(p >= s[0]).long() + (p >= s[0] + s[1]).long()].t()
    else:
        at = pos.double().reshape(-1, 1)
    a = at * freq
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    x = x.float()
    u, w = (x[..., :half], x[..., half:]) if c["neox"] else (x[..., 0::2], x[..., 1::2])
    y, z = u * cos - w * sin, u * sin + w * cos
    return torch.cat([y, z], -1) if c["neox"] else torch.stack([y, z], -1).flatten(-2)


def _plain_append(s):
    c = s["case"]
    b, i = _tokens(s)
    pos = s["pos"] if s["pos"] is not None else i[None]
    at, row = s["pages"].long()[b, i // c["page"]], i % c["page"]
    s["pool"][at, 0, :, row] = _rotate(s["k"], pos, c).to(torch.bfloat16)
    s["pool"][at, 1, :, row] = s["v"].to(torch.bfloat16)
    return {"q": _rotate(s["q"], pos, c).to(s["q"].dtype), "pool": s["pool"]}


def _plain_attention(s):
    c = s["case"]
    Hkv, hd, page = c["kv_heads"], c["head_dim"], c["page"]
    G = c["heads"] // Hkv
    b, i = _tokens(s)
    B, T, L = c["seqs"], max(_new(c)), max(_lens(c))
    # tokens and entries in padded batches
    first = torch.searchsorted(b, torch.arange(B, device="cuda"))
    t = torch.arange(b.numel(), device="cuda") - first[b]
    q = torch.zeros((B, T, c["heads"], hd), dtype=torch.float32, device="cuda")
    q[b, t] = s["q"].float()
    last = torch.full((B, T), -1, dtype=torch.int64, device="cuda")
    last[b, t] = i
    j = torch.arange(L, device="cuda")
    held = j < s["lens"].long()[:, None]
    at = torch.where(held, s["pages"].long()[:, j // page], torch.zeros((), dtype=torch.int64, device="cuda"))
    k, v = (s["pool"][at, n, :, j % page].transpose(1, 2).float() for n in (0, 1))
    rows = q.reshape(B, T, Hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, hd)
    x = torch.matmul(rows, k.transpose(2, 3)).mul_(hd ** -0.5)
    out_of = j > last[..., None]
    if c["window"]:
        out_of |= j <= last[..., None] - c["window"]
    x.masked_fill_(out_of.repeat_interleave(G, dim=1)[:, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    p.div_(p.sum(-1, keepdim=True).clamp(min=1e-38))
    o = torch.matmul(p, v).reshape(B, Hkv, T, G, hd).permute(0, 2, 1, 3, 4).reshape(B, T, c["heads"], hd)
    return {"out": o[b, t].to(s["q"].dtype)}


# ------------------------------------------------------------- measured calls
def prepare(case, seed):
    d = _inputs(case, seed)
    s = {"case": case, **{n: d.get(n) for n in ("q", "k", "v", "pos", "lens", "pages", "start", "group_start", "prefix")}}
    if own:
        import transformer_decode_step_gb300 as pnb

        s["kv"] = pnb.PagedKv(n_layer=1, n_head=case["heads"], n_kv_head=case["kv_heads"],
                              head_dim=case["head_dim"], n_page=d["n_page"], page=case["page"],
                              rope_theta=case["theta"], rope_neox=case["neox"],
                              rope_sections=_sections(case) if case["axes"] == 3 else None,
                              shared_tok=s["q"].shape[0] if case["op"] == "shared" else 0)
        s["kv"].pages(0).copy_(d["pool"])
        s["batch"] = s["kv"].batch(s["lens"], s["pages"], s["start"])
        s["out"] = torch.zeros_like(s["q"])
    else:
        s["pool"] = d["pool"]
    return s


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return _plain_append(s) if op == "append" else _plain_attention(s)
    if op == "append":
        s["kv"].append(0, s["batch"], s["k"], s["v"], q=s["q"], q_out=s["out"], pos=s["pos"])
        return {"q": s["out"], "pool": s["kv"].pages(0)}
    if op == "shared":
        s["kv"].attention_shared(0, s["batch"], s["group_start"], s["prefix"], s["q"], s["out"],
                                 window=s["case"]["window"])
    else:
        s["kv"].attention(0, s["batch"], s["q"], s["out"], window=s["case"]["window"])
    return {"out": s["out"]}


def work(case):
    c = case
    H, Hkv, hd, W = c["heads"], c["kv_heads"], c["head_dim"], c["window"]
    es = 4 if c["dtype"] == "fp32" else 2
    new, lens = _new(c), _lens(c)
    n_tok = sum(new)
    if c["op"] == "append":
        return {"bytes": n_tok * hd * (es * (2 * H + 2 * Hkv) + 4 * Hkv), "flops": 3 * n_tok * (H + Hkv) * hd}
    pairs = held = 0
    each = c["seqs"] // c["groups"] if c["groups"] else 1
    for b, (n, m) in enumerate(zip(new, lens)):
        # row t attends to entries up to m - n + t
        pairs += sum(min(m - n + t + 1, W or m) for t in range(n))
        low = max(0, m - n - W + 1) if W else 0
        own_from = _prefix(c)[b // each] if c["groups"] else 0
        held += m - max(low, own_from)
        if c["groups"] and b % each == 0:
            lows = [max(0, lens[x] - new[x] - W + 1) if W else 0 for x in range(b, b + each)]
            held += max(0, own_from - min(lows))
    return {"bytes": held * Hkv * hd * 4 + 2 * n_tok * H * hd * es, "flops": 4 * H * hd * pairs}


# ---------------------------------------------------------- in 64 bits
def exact(case, seed):
    c, d = case, _inputs(case, seed)
    H, Hkv, hd, page, W = c["heads"], c["kv_heads"], c["head_dim"], c["page"], c["window"]
    G = H // Hkv
    new, lens = _new(c), _lens(c)
    if c["op"] == "append":
        pool = d["pool"].double()
        out = torch.empty((sum(new), H, hd), dtype=torch.float64, device="cuda")
        axis = sum(([a] * n for a, n in enumerate(_sections(c))), [])
        done = 0
        for b, (n, m) in enumerate(zip(new, lens)):
            e = torch.arange(m - n, m, device="cuda")
            angle = torch.empty((n, 1, hd // 2), dtype=torch.float64, device="cuda")
            for p in range(hd // 2):
                at = e if d.get("pos") is None else d["pos"][axis[p], done:done + n]
                angle[:, 0, p] = at.double() / c["theta"] ** (2 * p / hd)
            turn = torch.polar(torch.ones_like(angle), angle)
            for name in "qk":
                x = d[name][done:done + n].double()
                if c["neox"]:
                    x = x.unflatten(-1, (2, -1)).transpose(-1, -2).contiguous()
                    y = torch.view_as_real(torch.view_as_complex(x) * turn).transpose(-1, -2).flatten(-2)
                else:
                    y = torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
                if name == "q":
                    out[done:done + n] = y
                else:
                    pool[d["pages"][b].long()[e // page], 0, :, e % page] = y
            pool[d["pages"][b].long()[e // page], 1, :, e % page] = d["v"][done:done + n].double()
            done += n
        return {"q": out, "pool": pool}
    out = torch.empty((sum(new), H, hd), dtype=torch.float64, device="cuda")
    done = 0
    for b, (n, m) in enumerate(zip(new, lens)):
        rows = d["pool"][d["pages"][b, :-(-m // page)].long()]          # [pages][2][Hkv][page][hd]
        k, v = (rows[:, x].permute(1, 0, 2, 3).reshape(Hkv, -1, hd)[:, :m] for x in (0, 1))
        for t in range(0, n, 512):
            u = min(n, t + 512)
            lo, hi = max(0, m - n + t - W + 1) if W else 0, m - n + u
            e = torch.arange(lo, hi, device="cuda")
            own_e = torch.arange(m - n + t, hi, device="cuda")[:, None]
            see = (e <= own_e) & ((e > own_e - W) if W else True)
            for h in range(Hkv):
                q = d["q"][done + t:done + u, h * G:(h + 1) * G].double().permute(1, 0, 2)
                z = (q @ k[h, lo:hi].double().t()) / hd ** 0.5
                z = torch.where(see, z, -math.inf)
                out[done + t:done + u, h * G:(h + 1) * G] = (torch.softmax(z, -1) @ v[h, lo:hi].double()).permute(1, 0, 2)
        done += n
    return {"out": out}
