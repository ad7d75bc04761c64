"""The paged KV cache on the GPU against a plain implementation in 64 bits.

Every pool row that holds no entry of a case is NaN, page tables name nonsense behind a
sequence's last page, and rows behind the last sequence must stay as they are.

Tolerances (u = 2^-8, the half step of bf16; A the largest sum |q_i k_i| / sqrt(head_dim) of a
pair; V the largest |value|):
  * with fp32 on either side queries and weights are two bf16 numbers, off by at most u^2 = 2^-16
    of the value, so scores by A 2^-16 (and the fp32 sums' A hd 2^-24), weights by that and 2^-16,
    and the weighted mean, whose weights' sum is off by as much, by twice their sum times V;
  * with bf16 on both sides the weights are off by u at most and the output by u more: 2 u V
    beside the same terms of the scores (their products are exact, only the sums round).
"""
import math

import pytest
import torch

import transformer_decode_step_gb300 as pnb

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -8


class Case:
    """A pool, page tables and lengths; entries[b] = (K, V) in [len][n_kv][hd] bf16 on the GPU."""

    def __init__(self, lens, n_kv=2, G=2, hd=128, page=32, seed=0, new=None, prefix=None, k_scale=1.0, extra_pages=3,
                 max_page=None, n_layer=1, **kw):
        self.lens, self.n_kv, self.G, self.hd, self.page, self.H = lens, n_kv, G, hd, page, n_kv * G
        self.new = [1] * len(lens) if new is None else new
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.gen = gen
        B = len(lens)
        prefix = prefix or [(list(range(B)), 0)]
        need = [-(-n // page) for n in lens]
        self.max_page = max_page or max(need + [1]) + 1
        self.n_page = sum(need) + extra_pages
        order = torch.randperm(self.n_page, generator=gen, device="cuda").tolist()
        self.kv = pnb.PagedKv(n_layer=n_layer, n_head=self.H, n_kv_head=n_kv, head_dim=hd, n_page=self.n_page, page=page,
                              **kw)
        pool = self.kv.pages(0)
        pool.fill_(float("nan"))
        table = torch.full((B, self.max_page), 1 << 30, dtype=torch.int32)
        table[:, 1::2] = -5
        at = 0
        self.entries = [None] * B
        for group, shared in prefix:
            lead = group[0]
            for b in group:
                first = shared // page if b != lead else 0
                if first:
                    table[b, :first] = table[lead, :first]
                for i in range(first, need[b]):
                    table[b, i] = order[at]
                    at += 1
                rows = []
                for s in (k_scale, 1.0):
                    x = (torch.randn((lens[b], n_kv, hd), generator=gen, device="cuda") * s).to(torch.bfloat16)
                    rows.append(x)
                if first:
                    for x, y in zip(rows, self.entries[lead]):
                        x[:first * page] = y[:first * page]
                self.entries[b] = tuple(rows)
        self.table_cpu = table
        self.table = table.cuda()
        for b in range(B):
            self.store(b)
        self.len_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        starts = [0]
        for n in self.new:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.start_t = torch.tensor(starts, dtype=torch.int32, device="cuda")

    def store(self, b):
        pool = self.kv.pages(0)
        if self.lens[b] == 0:
            return
        e = torch.arange(self.lens[b], device="cuda")
        ids = self.table[b].long()[e // self.page]
        for s in (0, 1):
            pool[ids, s, :, e % self.page] = self.entries[b][s]

    def queries(self, dtype, scale=1.0, tail=0):
        return (torch.randn((self.starts[-1] + tail, self.H, self.hd), generator=self.gen, device="cuda") * scale).to(DT[dtype])

    def batch(self, ragged=True):
        return self.kv.batch(self.len_t, self.table, self.start_t if ragged else None)

    def want(self, q, window=0):
        """(out, A, V) in 64 bits."""
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        most = big = 0.0
        for b, (n, m) in enumerate(zip(self.new, self.lens)):
            if n == 0 or m == 0:
                continue
            k, v = (x.double().transpose(0, 1) for x in self.entries[b])       # [n_kv][m][hd]
            rows = q[self.starts[b]:self.starts[b + 1]].double().unflatten(1, (self.n_kv, self.G))   # [n][kv][G][hd]
            s = torch.einsum("tkgd,kmd->tkgm", rows, k) / math.sqrt(self.hd)
            most = max(most, float(torch.einsum("tkgd,kmd->tkgm", rows.abs(), k.abs()).max()) / math.sqrt(self.hd))
            big = max(big, float(v.abs().max()))
            i = torch.arange(m - n, m, device="cuda")[:, None]
            j = torch.arange(m, device="cuda")
            see = (j <= i) & ((j > i - window) if window else torch.ones_like(j <= i))
            s = torch.where(see[:, None, None], s, torch.full_like(s, -math.inf))
            p = torch.softmax(s, -1)
            p = torch.where(see.any(-1)[:, None, None, None], p, torch.zeros_like(p))
            out[self.starts[b]:self.starts[b + 1]] = torch.einsum("tkgm,kmd->tkgd", p, v).flatten(1, 2)
        return out, most, big

    def check(self, got, q, window=0, tail=0):
        n = self.starts[-1]
        want, A, V = self.want(q[:n], window)
        assert torch.isfinite(got[:n].double()).all()
        exact = q.dtype == torch.float32 or got.dtype == torch.float32
        score = A * (2.0 ** -16 + self.hd * 2.0 ** -24)
        tol = 2 * (score + 2.0 ** -16 + 2.0 ** -18) * V + (0 if exact else U * V)
        if got.dtype == torch.bfloat16:
            tol += U * V
        err = float((got[:n].double() - want).abs().max()) if n else 0.0
        assert err <= tol, (err, tol)
        if tail:
            assert bool((got[n:] == 7).all())
        assert self.kv.device_error() == 0

    def run(self, dtype, out_dtype=None, window=0, ragged=True, scale=1.0, tail=0):
        q = self.queries(dtype, scale, tail)
        out = torch.full(q.shape, 7.0, dtype=DT[out_dtype or dtype], device="cuda")
        self.kv.attention(0, self.batch(ragged), q, out, window=window)
        self.check(out, q, window, tail)
        return q, out


# ----------------------------------------------------------------- append
def _rotate64(x, pos, theta, neox, sections):
    """x [n][heads][hd]; pos [axes][n]."""
    hd = x.shape[-1]
    x = x.double()
    y = x.clone()
    ends = [sum(sections[:i + 1]) for i in range(len(sections))]
    for p in range(hd // 2):
        axis = next(a for a, e in enumerate(ends) if p < e)
        ang = pos[axis].double() * theta ** (-2.0 * p / hd)
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        i, j = (p, p + hd // 2) if neox else (2 * p, 2 * p + 1)
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def _near_rotated(got, want, x, half_step):
    """cos and sin are off by pi 2^-24 for the angle's rounding and 2^-23 for their own, products and sum by
    2^-24 each: below 2^-21 of the pair's magnitudes, and the result's rounding."""
    tol = 2 * x.double().abs().amax(-1, keepdim=True) * 2.0 ** -21 + want.abs() * half_step
    assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("neox", [False, True])
@pytest.mark.parametrize("dtype,hd,page,n_kv,G,new,old,axes", [
    ("bf16", 128, 64, 2, 4, [1, 1, 1, 1], [5, 63, 64, 127], 1),
    ("fp32", 64, 16, 1, 3, [7, 0, 33, 1], [0, 4, 15, 100], 1),
    ("fp32", 128, 32, 5, 1, [40, 3], [0, 31], 3),
    ("bf16", 64, 128, 4, 2, [129, 2, 0], [0, 126, 0], 3),
    ("bf16", 128, 16, 8, 4, [1300], [3], 1),
])
def test_append(neox, dtype, hd, page, n_kv, G, new, old, axes):
    lens = [n + o for n, o in zip(new, old)]
    sections = [hd // 8, hd // 16 * 3, hd // 16 * 3] if axes == 3 else None
    theta = 500000.0
    c = Case(lens, n_kv, G, hd, page, seed=1, new=new, rope_theta=theta, rope_neox=neox, rope_sections=sections)
    before = c.kv.pages(0).clone()
    n = c.starts[-1]
    gen = c.gen
    rows = lambda h: torch.randn((n + 2, h, hd), generator=gen, device="cuda").to(DT[dtype])  # noqa: E731
    q, k, v = rows(c.H), rows(n_kv), rows(n_kv)
    pos = torch.randint(0, 1 << 20, (3, n + 2) if axes == 3 else (n + 2,), generator=gen, device="cuda", dtype=torch.int32)
    use_pos = axes == 3 or hd == 64
    q_out = torch.full_like(q, 7.0)
    c.kv.append(0, c.batch(), k, v, q=q, q_out=q_out, pos=pos if use_pos else None)
    entry = torch.cat([torch.arange(m - a, m) for a, m in zip(new, lens)]).cuda()
    at = pos[..., :n].reshape(axes, n) if use_pos else entry[None]
    half = 0.0 if dtype == "fp32" else U
    wq = _rotate64(q[:n], at, theta, neox, sections or [hd // 2])
    _near_rotated(q_out[:n], wq, q[:n], half)
    assert bool((q_out[n:] == 7).all())
    wk = _rotate64(k[:n], at, theta, neox, sections or [hd // 2])
    after = c.kv.pages(0)
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
    ids = c.table.long()[seq, entry // page]
    _near_rotated(after[ids, 0, :, entry % page], wk, k[:n], U)
    assert torch.equal(after[ids, 1, :, entry % page], v[:n].to(torch.bfloat16))
    keep = torch.ones(before.shape[0], page, dtype=torch.bool, device="cuda")
    keep[ids, entry % page] = False
    a, b = (x.view(torch.int16).permute(0, 3, 1, 2, 4)[keep] for x in (after, before))
    assert torch.equal(a, b)
    assert c.kv.device_error() == 0


def test_append_in_place_fused_projection():
    # q, k and v side by side in one projection's rows, queries rotated where they lie
    hd, n_kv, G, n = 128, 2, 4, 37
    c = Case([n + 5], n_kv, G, hd, 32, seed=2, new=[n], rope_theta=10000.0)
    qkv = torch.randn((n, (c.H + 2 * n_kv) * hd), generator=c.gen, device="cuda")
    x = qkv.clone().view(n, -1, hd)
    q, k, v = x[:, :c.H], x[:, c.H:c.H + n_kv], x[:, c.H + n_kv:]
    c.kv.append(0, c.batch(), k, v, q=q)
    at = torch.arange(5, n + 5, device="cuda")[None]
    y = qkv.view(n, -1, hd)
    _near_rotated(q, _rotate64(y[:, :c.H], at, 10000.0, False, [64]), y[:, :c.H], 0.0)
    assert torch.equal(k, y[:, c.H:c.H + n_kv]) and torch.equal(v, y[:, c.H + n_kv:])


def test_append_without_rotation_and_without_queries():
    c = Case([20, 9], 2, 2, 64, 16, seed=3, new=[20, 4], rope_theta=0.0)
    k = torch.randn((24, 2, 64), generator=c.gen, device="cuda")
    v = torch.randn((24, 2, 64), generator=c.gen, device="cuda").to(torch.float32)
    c.kv.append(0, c.batch(), k, v)
    e = torch.cat([torch.arange(20), torch.arange(5, 9)]).cuda()
    ids = c.table.long()[torch.tensor([0] * 20 + [1] * 4, device="cuda"), e // 16]
    assert torch.equal(c.kv.pages(0)[ids, 0, :, e % 16], k.to(torch.bfloat16))
    assert torch.equal(c.kv.pages(0)[ids, 1, :, e % 16], v.to(torch.bfloat16))


def test_append_far_and_negative_positions():
    c = Case([4], 1, 1, 128, 16, seed=4, new=[4], rope_theta=10000.0)
    pos = torch.tensor([(1 << 31) - 1, 123456789, -7, -(1 << 31)], dtype=torch.int32, device="cuda")
    k = torch.randn((4, 1, 128), generator=c.gen, device="cuda")
    q, out = k.clone(), torch.empty_like(k)
    c.kv.append(0, c.batch(), k, k, q=q, q_out=out, pos=pos)
    # the powers of theta are rounded to double, 2^-53 of them, times a position: 2^-21 of a radian, in
    # either result, the logarithm's and the exponential's roundings in `pow` up to as much again
    want = _rotate64(q, pos[None], 10000.0, False, [64])
    tol = q.double().abs().amax(-1, keepdim=True) * 2 * (2.0 ** -21 + 4 * 2.0 ** -21)
    assert bool(((out.double() - want).abs() <= tol).all())


def test_append_drops_what_has_no_entry():
    # sequence 0 lies behind its page table, sequence 1 has more tokens than entries, sequence 2's page is nonsense
    c = Case([16, 16, 16, 16], 1, 1, 64, 16, seed=5, new=[2, 3, 1, 1], max_page=2, rope_theta=0.0)
    before = c.kv.pages(0).clone()
    c.len_t.copy_(torch.tensor([33, 2, 16, 16]))
    c.table[2, 0] = c.n_page
    k = torch.randn((7, 1, 64), generator=c.gen, device="cuda")
    c.kv.append(0, c.batch(), k, k)
    want = before
    # sequence 0: entries 31 (a nonsense page) and 32 (no page); sequence 1: entries -1, 0 and 1
    for t, e in ((3, 0), (4, 1)):
        want[c.table[1, 0].long(), :, :, e] = k[t].to(torch.bfloat16)
    want[c.table[3, 0].long(), :, :, 15] = k[6].to(torch.bfloat16)
    assert torch.equal(c.kv.pages(0).view(torch.int16), want.view(torch.int16))
    assert c.kv.device_error() == pnb.PNB_DEV_ERR_FULL | pnb.PNB_DEV_ERR_RANGE
    assert c.kv.device_error() == 0


# -------------------------------------------------------------- attention
PROMPTS = [
    # lens, new, n_kv, G, hd, page
    ([1], [1], 1, 1, 64, 16),
    ([13], [13], 4, 2, 64, 16),
    ([128, 0, 257, 1, 30], [128, 0, 257, 1, 7], 2, 4, 128, 64),
    ([700], [700], 1, 8, 128, 128),
    ([129, 640], [1, 200], 1, 3, 128, 16),
    ([511, 1025, 90], [511, 1025, 90], 2, 1, 64, 32),
    ([2049], [65], 1, 5, 128, 32),
    ([3, 5, 7, 300], [2, 5, 1, 299], 2, 7, 64, 128),
    ([1100], [40], 1, 64, 64, 64),
    ([4500, 1], [128, 1], 5, 1, 128, 16),
]


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("lens,new,n_kv,G,hd,page", PROMPTS)
def test_attention_packed(lens, new, n_kv, G, hd, page, dtype, out_dtype):
    Case(lens, n_kv, G, hd, page, seed=11, new=new).run(dtype, out_dtype, tail=3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window", [1, 2, 63, 128, 129, 300, 5000])
def test_attention_window(window, dtype):
    Case([700, 10, 333], 2, 2, 128, 32, seed=12, new=[700, 10, 3]).run(dtype, window=window)
    Case([700, 400], 2, 2, 64, 64, seed=13).run(dtype, window=window, ragged=False)


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("lens,T,n_kv,G,hd,page", [
    ([1, 2, 3, 700, 128, 129], 1, 2, 4, 128, 64),
    ([5000], 1, 1, 1, 128, 16),
    ([9000], 1, 8, 8, 64, 128),
    ([300] * 70, 1, 2, 7, 64, 32),
    ([40, 1000, 5], 5, 2, 4, 128, 16),
    ([6000], 2, 4, 4, 128, 32),
    ([0, 33], 1, 1, 2, 128, 16),
    ([777, 12], 3, 1, 16, 64, 64),
])
def test_attention_steps(lens, T, n_kv, G, hd, page, dtype, out_dtype):
    Case(lens, n_kv, G, hd, page, seed=14, new=[T] * len(lens)).run(dtype, out_dtype, ragged=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_many_sequences(dtype):
    g = torch.Generator()
    g.manual_seed(5)
    lens = torch.randint(0, 60, (1024,), generator=g).tolist()
    new = [min(n, int(x)) for n, x in zip(lens, torch.randint(0, 4, (1024,), generator=g))]
    Case(lens, 1, 2, 64, 16, seed=15, new=new).run(dtype, tail=1)
    Case(lens, 1, 2, 64, 16, seed=15).run(dtype, ragged=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("new", [[1], [600]])
def test_attention_large_and_growing_scores(dtype, new):
    # scores that grow by hundreds along the sequence: the reference of the sums moves in every tile
    c = Case([1500], 1, 4, 128, 64, seed=16, new=new)
    k = c.entries[0][0]
    k.copy_((k.float() * torch.linspace(0.01, 30, 1500, device="cuda")[:, None, None]).to(torch.bfloat16))
    c.store(0)
    c.run(dtype, scale=3.0, ragged=len(new) > 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,G,hd", [(32, 4, 128), (5, 4, 128), (128, 1, 64), (40, 3, 64), (9, 1, 128)])
@pytest.mark.parametrize("window", [0, 30, 100, 500])
def test_blocks_of_few_rows(T, G, hd, window, dtype):
    # windows begin at every place within a tile, and references move in some warps and not in others
    lens = [700 + 37 * i for i in range(12)]
    c = Case(lens, 2, G, hd, 32, seed=17, new=[T] * len(lens))
    for b, n in enumerate(lens):
        k = c.entries[b][0]
        k.copy_((k.float() * torch.linspace(0.01, 4, n, device="cuda")[:, None, None]).to(torch.bfloat16))
        c.store(b)
    c.run(dtype, window=window, scale=2.0, ragged=False)


@pytest.mark.parametrize("T", [1, 3, 40])
def test_more_tokens_than_entries_answer_zero(T):
    c = Case([2, 0, 200], 2, 2, 64, 16, seed=17, new=[T] * 3)
    q = c.queries("fp32")
    out = torch.full_like(q, 7.0)
    c.kv.attention(0, c.batch(False), q, out)
    want, A, V = c.want(q)
    assert float((out.double() - want).abs().max()) <= 2 * (A * 2.0 ** -15 + 2.0 ** -15) * V
    for b in range(3):
        dead = max(0, T - c.lens[b])
        assert bool((out[c.starts[b]:c.starts[b] + dead] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("new,bad", [([300], 250), ([5], 297), ([300], 3)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_a_row_does_not_see(new, bad, value, dtype):
    # a NaN or an infinity among the values reaches the rows that attend to it, and no others
    c = Case([300], 2, 2, 128, 32, seed=18, new=new)
    c.entries[0][1][bad] = value
    c.entries[0][0][bad, 1] = float("nan")
    c.store(0)
    q = c.queries(dtype)
    out = torch.full_like(q, 7.0)
    window = 40
    for w in (0, window):
        c.kv.attention(0, c.batch(), q, out, window=w)
        i = torch.arange(300 - new[0], 300, device="cuda")
        sees = (bad <= i) & ((bad > i - w) if w else torch.ones_like(i, dtype=torch.bool))
        assert not bool(torch.isfinite(out[sees]).any())
        clean = Case.__new__(Case)
        clean.__dict__.update(c.__dict__)
        clean.entries = [tuple(torch.where(torch.isfinite(x), x, torch.zeros_like(x)) for x in c.entries[0])]
        want, A, V = clean.want(q, w)
        tol = 2 * (A * 2.0 ** -15 + 2.0 ** -15) * V + (2 * U * V if dtype == "bf16" else 0)
        diff = (out.double() - want)[~sees]
        assert diff.numel() == 0 or float(diff.abs().max()) <= tol


# ----------------------------------------------------------------- shared
SHARED = [
    # groups of (sequences, prefix), entries behind it, T, n_kv, G, hd, page
    ([([0, 1, 2, 3], 64)], [1, 5, 0, 40], 1, 2, 4, 128, 64),
    ([([0, 1, 2, 3, 4], 512)], [1, 200, 30, 7, 16], 1, 1, 8, 64, 16),
    ([([0, 1], 96), ([2], 1024), ([3, 4, 5], 32)], [3, 300, 1, 2, 129, 64], 2, 2, 3, 128, 32),
    ([([0], 0), ([1, 2], 128)], [10, 1, 500], 1, 2, 7, 64, 128),
    ([(list(range(40)), 2048)], [(i * 37) % 150 for i in range(40)], 1, 2, 8, 128, 64),
    ([(list(range(20)), 1024), (list(range(20, 33)), 512)], [(i * 29) % 400 for i in range(33)], 5, 1, 4, 128, 16),
    ([(list(range(64)), 8192)], [i % 9 for i in range(64)], 1, 1, 4, 64, 128),
    ([([0, 1], 20000)], [1000, 3], 1, 4, 1, 128, 32),
]


def _wide(n_seq, n_kv, hd, page):
    """Page tables wide enough for the prefix to be attended once per group (small batches go
    sequence by sequence)."""
    return -(-(1 << 29) // (n_seq * page * n_kv * hd * 4))


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "fp32")])
@pytest.mark.parametrize("groups,own,T,n_kv,G,hd,page", SHARED)
@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("wide", [True, False])
def test_shared(groups, own, T, n_kv, G, hd, page, wide, window, dtype, out_dtype):
    pre = [0] * len(own)
    for seqs, p in groups:
        for b in seqs:
            pre[b] = p
    lens = [p + o + T for p, o in zip(pre, own)]
    c = Case(lens, n_kv, G, hd, page, seed=21, new=[T] * len(own), prefix=[(s, p // page * page) for s, p in groups],
             shared_tok=len(own) * T, max_page=_wide(len(own), n_kv, hd, page) if wide else None)
    q = c.queries(dtype)
    out = torch.full(q.shape, 7.0, dtype=DT[out_dtype], device="cuda")
    start = torch.tensor([s[0] for s, _ in groups] + [len(own)], dtype=torch.int32, device="cuda")
    prefix = torch.tensor([p for _, p in groups], dtype=torch.int32, device="cuda")
    c.kv.attention_shared(0, c.batch(False), start, prefix, q, out, window=window)
    c.check(out, q, window)


def test_shared_prefix_that_covers_whole_sequences():
    # the prefix reaches past some sequences' queries: what a row does not see stays unseen
    c = Case([200, 200, 210], 2, 2, 64, 16, seed=22, new=[4, 4, 4], prefix=[([0, 1, 2], 192)], shared_tok=12,
             max_page=_wide(3, 2, 64, 16))
    q = c.queries("fp32")
    out = torch.full_like(q, 7.0)
    start = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    for p in (0, 16, 180, 192, 199):
        prefix = torch.tensor([p], dtype=torch.int32, device="cuda")
        c.kv.attention_shared(0, c.batch(False), start, prefix, q, out)
        c.check(out, q)


def test_shared_pages_written_by_the_step_itself():
    # drafted tokens of a single sequence inside its "prefix"
    c = Case([64], 1, 2, 64, 16, seed=23, new=[8], shared_tok=8, max_page=_wide(1, 1, 64, 16))
    q = c.queries("fp32")
    out = torch.full_like(q, 7.0)
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    c.kv.attention_shared(0, c.batch(False), one, torch.tensor([64], dtype=torch.int32, device="cuda"), q, out)
    c.check(out, q)


# --------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_serving_run(dtype):
    """A system prompt once, four requests behind it in its pages, a chunk each, then decode steps: every
    answer against attention in 64 bits over the rotated rows that the cache was given."""
    hd, n_kv, G, page, sys_n = 128, 2, 4, 32, 160
    H, B, layers = n_kv * G, 4, 2
    kv = pnb.PagedKv(n_layer=layers, n_head=H, n_kv_head=n_kv, head_dim=hd, n_page=64, page=page, shared_tok=B)
    kv.buf.fill_(255)   # NaN
    gen = torch.Generator(device="cuda")
    gen.manual_seed(31)
    table = torch.zeros((B, _wide(B, n_kv, hd, page)), dtype=torch.int32)
    table[:, :5] = torch.tensor([7, 3, 60, 21, 9])
    for b in range(B):
        table[b, 5:12] = 22 + 7 * b + torch.arange(7)
    table = table.cuda()
    held = [[[[], []] for _ in range(B)] for _ in range(layers)]

    def rows(n):
        return [torch.randn((n, h, hd), generator=gen, device="cuda").to(DT[dtype]) for h in (H, n_kv, n_kv)]

    def tokens(layer, batch, new, lens, shared=None):
        q, k, v = rows(sum(new))
        seqs = list(range(len(new)))
        rot = torch.empty_like(q)
        kv.append(layer, batch, k, v, q=q, q_out=rot)
        out = torch.full_like(q, 7.0)
        if shared is None:
            kv.attention(layer, batch, rot, out)
        else:
            kv.attention_shared(layer, batch, *shared, rot, out)
        at = 0
        for b in seqs:
            n, e = new[b], torch.arange(lens[b] - new[b], lens[b], device="cuda")
            if n == 0:
                continue
            kr = _rotate64(k[at:at + n], e[None], 10000.0, False, [hd // 2]).to(torch.bfloat16)
            held[layer][b][0].append(kr)
            held[layer][b][1].append(v[at:at + n].to(torch.bfloat16))
            kk, vv = (torch.cat(x).double().transpose(0, 1) for x in held[layer][b])
            qq = rot[at:at + n].double().unflatten(1, (n_kv, G))
            s = torch.einsum("tkgd,kmd->tkgm", qq, kk) / math.sqrt(hd)
            A = float(torch.einsum("tkgd,kmd->tkgm", qq.abs(), kk.abs()).max()) / math.sqrt(hd)
            see = torch.arange(lens[b], device="cuda") <= e[:, None]
            p = torch.softmax(torch.where(see[:, None, None], s, torch.full_like(s, -math.inf)), -1)
            want = torch.einsum("tkgm,kmd->tkgd", p, vv).flatten(1, 2)
            V = float(vv.abs().max())
            # a key within 2^-20 of a rounding border may be held as its neighbour, 2^-7 of it away: that
            # moves one of head_dim products of a score
            edge = 2 * 2.0 ** -7 * float(qq.abs().max() * kk.abs().max()) / math.sqrt(hd) * V
            tol = 2 * (A * 2.0 ** -15 + 2.0 ** -15) * V + edge + (2 * U * V if dtype == "bf16" else 0)
            assert float((out[at:at + n].double() - want).abs().max()) <= tol
            at += n

    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = [sys_n] * B
    for layer in range(layers):     # the system prompt, in the pages that all requests name
        tokens(layer, kv.batch(ints(sys_n), table[:1].contiguous()), [sys_n], [sys_n])
        for b in range(1, B):
            held[layer][b] = [list(x) for x in held[layer][0]]
    new = [30, 1, 0, 77]
    lens = [a + n for a, n in zip(lens, new)]
    for layer in range(layers):
        tokens(layer, kv.batch(ints(*lens), table, ints(0, 30, 31, 31, 108)), new, lens)
    for _ in range(3):
        lens = [n + 1 for n in lens]
        for layer in range(layers):
            tokens(layer, kv.batch(ints(*lens), table), [1] * B, lens, (ints(0, B), ints(sys_n)))
    assert kv.device_error() == 0


def test_captured_calls_follow_the_device_tensors():
    c = Case([300, 77], 2, 4, 128, 32, seed=41, new=[5, 5], prefix=[([0, 1], 64)], shared_tok=10,
             max_page=_wide(2, 2, 128, 32))
    q = c.queries("bf16")
    out, out2 = torch.zeros_like(q), torch.zeros_like(q)
    start = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    prefix = torch.tensor([64], dtype=torch.int32, device="cuda")
    b = c.batch(False)
    ragged = c.batch()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.kv.attention(0, ragged, q, out)
        c.kv.attention_shared(0, b, start, prefix, q, out2)
    torch.cuda.current_stream().wait_stream(side)
    c.check(out, q)
    c.check(out2, q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.kv.attention(0, ragged, q, out)
        c.kv.attention_shared(0, b, start, prefix, q, out2)
    for lens, new in (([290, 70], [5, 5]), ([300, 66], [5, 5])):
        c.lens, c.new = lens, new
        c.len_t.copy_(torch.tensor(lens))
        c.entries = [tuple(x[:n] for x in e) for e, n in zip(c.entries, lens)] if lens[0] < 300 else c.entries
        if lens[0] == 300:
            d = Case([300, 66], 2, 4, 128, 32, seed=41, new=new, prefix=[([0, 1], 64)], shared_tok=10)
            c.kv.pages(0).copy_(d.kv.pages(0)[:c.n_page] if d.n_page >= c.n_page else
                                torch.cat([d.kv.pages(0), c.kv.pages(0)[d.n_page:]]))
            c.table.fill_(-1)
            c.table[:, :d.table.shape[1]] = d.table
            c.entries = d.entries
        q.copy_(c.queries("bf16"))
        out.fill_(7.0)
        out2.fill_(7.0)
        g.replay()
        c.check(out, q)
        c.check(out2, q)


@pytest.mark.parametrize("new", [[1] * 6, [400, 1, 33, 0, 128, 900]])
def test_same_bits_every_time(new):
    lens = [n + 2000 * (i % 3) for i, n in enumerate(new)]
    c = Case(lens, 2, 4, 128, 64, seed=42, new=new)
    q = c.queries("bf16")
    outs = []
    for _ in range(4):
        out = torch.zeros_like(q)
        c.kv.attention(0, c.batch(), q, out)
        outs.append(out)
    for o in outs[1:]:
        assert torch.equal(outs[0].view(torch.int16), o.view(torch.int16))


def test_two_caches_on_two_streams():
    cs = [Case([900, 50], 2, 4, 128, 32, seed=s, new=[900, 3]) for s in (43, 44)]
    qs = [c.queries("bf16") for c in cs]
    outs = [torch.zeros_like(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, q, o, s in zip(cs, qs, outs, streams):
            with torch.cuda.stream(s):
                c.kv.attention(0, c.batch(), q, o)
    torch.cuda.synchronize()
    for c, q, o in zip(cs, qs, outs):
        c.check(o, q)


def test_strided_rows_and_in_place():
    # queries inside a fused projection's rows, answers over them
    hd, n_kv, G, n = 64, 2, 2, 50
    c = Case([n + 7], n_kv, G, hd, 16, seed=45, new=[n])
    x = torch.randn((n, c.H + 2 * n_kv, hd), generator=c.gen, device="cuda")
    keep = x.clone()
    q = x[:, :c.H]
    want = keep[:, :c.H].clone()
    c.kv.attention(0, c.batch(), q, q)
    c.check(q, want)
    assert torch.equal(x[:, c.H:], keep[:, c.H:])
    # heads outside tokens
    y = torch.empty((c.H, n, hd), device="cuda")
    c.kv.attention(0, c.batch(), want, y.transpose(0, 1))
    c.check(y.transpose(0, 1), want)


def test_offsets_past_32_bits():
    # 40000 pages of 128 entries, 2 x 64 x 128: five billion elements; the sequence lies in the last pages
    page, hd, n_page = 128, 128, 160000
    kv = pnb.PagedKv(n_layer=1, n_head=4, n_kv_head=1, head_dim=hd, n_page=n_page, page=page,
                     buf=torch.empty(n_page * 2 * page * hd * 2, dtype=torch.uint8, device="cuda"), rope_theta=0.0)
    n = 300
    gen = torch.Generator(device="cuda")
    gen.manual_seed(51)
    k, v = (torch.randn((n, 1, hd), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((n, 4, hd), generator=gen, device="cuda")
    table = torch.tensor([[n_page - 1, 0, n_page - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    b = kv.batch(lens, table)
    kv.append(0, b, k, v)
    assert torch.equal(kv.pages(0)[n_page - 1, 1, 0], v[:128, 0])
    s = torch.einsum("thd,md->htm", q.double(), k[:, 0].double()) / math.sqrt(hd)
    s = s.masked_fill(torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1), -math.inf)
    want = torch.einsum("htm,md->thd", torch.softmax(s, -1), v[:, 0].double())
    out = torch.empty_like(q)
    kv.attention(0, b, q, out)
    assert float((out.double() - want).abs().max()) <= 2e-3
    one = torch.empty((1, 4, hd), device="cuda")
    kv.attention(0, b, q[-1:].contiguous(), one)
    assert float((one.double() - want[-1:]).abs().max()) <= 2e-3


def test_nonsense_in_device_tensors_is_reported():
    c = Case([100, 40], 2, 2, 64, 16, seed=61, new=[3, 3], shared_tok=6, max_page=_wide(2, 2, 64, 16))
    q = c.queries("fp32")
    out = torch.zeros_like(q)
    start = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    prefix = torch.tensor([16], dtype=torch.int32, device="cuda")
    c.table[1, 1] = c.n_page + 3       # a page that is none
    for ragged in (True, False):
        c.kv.attention(0, c.batch(ragged), q, out)
        assert c.kv.device_error() == pnb.PNB_DEV_ERR_RANGE
    good = c.want(q)[0]
    assert float((out.double() - good)[:3].abs().max()) < 1e-2
    c.len_t.copy_(torch.tensor([-3, 1 << 30]))
    c.kv.attention(0, c.batch(), q, out)
    assert c.kv.device_error() == pnb.PNB_DEV_ERR_RANGE
    assert bool((out[:3] == 0).all())
    c.len_t.copy_(torch.tensor([100, 40]))
    for bad in ([0, 9, 6], [4, 2, 6], [-3, 3, 6], [0, 3, 1 << 20]):
        c.start_t.copy_(torch.tensor(bad))
        c.kv.attention(0, c.batch(), q, out)
        c.kv.append(0, c.batch(), torch.zeros((6, 2, 64), device="cuda"), torch.zeros((6, 2, 64), device="cuda"))
        c.kv.device_error()
    for gs, p in (([0, 5], 16), ([1, 2], 16), ([2, 0], 16), ([0, 2], 1 << 30), ([0, 2], -8)):
        start.copy_(torch.tensor(gs))
        prefix.fill_(p)
        c.kv.attention_shared(0, c.batch(False), start, prefix, q, out)
        c.kv.device_error()
    torch.cuda.synchronize()


# --------------------------------------------------------------- refusals
def test_refusals():
    c = Case([100, 40], 2, 2, 64, 16, seed=71, new=[3, 3], shared_tok=4)
    q = c.queries("fp32")
    out = torch.zeros_like(q)
    k = torch.zeros((6, 2, 64), device="cuda")
    b = c.batch()

    def refused(code, f, *a, **kw):
        with pytest.raises(pnb.PnbError) as e:
            f(*a, **kw)
        assert e.value.code == code

    refused(-1, c.kv.attention, 1, b, q, out)
    refused(-1, c.kv.attention, 0, b, q, out, window=-1)
    refused(-1, c.kv.attention, 0, b, q, out[:5])
    refused(-1, c.kv.attention, 0, b, q.half(), out)
    refused(-1, c.kv.attention, 0, b, q[..., ::2], out)
    refused(-1, c.kv.attention, 0, b, q, q[:1].expand(6, -1, -1))              # rows written over one another
    refused(-1, c.kv.attention, 0, c.batch(False), q[:5], out[:5])             # not a multiple of the sequences
    refused(-1, c.kv.attention_shared, 0, b, c.len_t.new_zeros(2), c.len_t.new_zeros(1), q[:4], out[:4])
    refused(-1, c.kv.attention_shared, 0, c.batch(False), c.len_t.new_zeros(2), c.len_t.new_zeros(1), q, out)
    refused(-1, c.kv.append, 0, b, k, k.bfloat16())
    refused(-1, c.kv.append, 0, b, k, k, q=q.bfloat16())
    refused(-1, c.kv.append, 0, b, k, k, q=q, q_out=out, pos=c.len_t)
    refused(-1, c.kv.append, 0, b, k, k, q_out=out)
    big = torch.zeros((6, 8, 64), device="cuda")
    refused(-1, c.kv.append, 0, b, big[:, 2:4], big[:, 6:], q=q, q_out=big[:, :4])   # over the keys
    inside = c.kv.buf[:6 * 2 * 64 * 4].view(torch.float32).view(6, 2, 64)
    refused(-1, c.kv.append, 0, b, inside, k)                                  # rows in the pool itself
    off = torch.zeros(6 * 4 * 64 + 1, device="cuda")[1:].view(6, 4, 64)
    refused(-3, c.kv.attention, 0, b, off, out)
    refused(-1, c.kv.batch, c.len_t.long(), c.table)
    refused(-1, c.kv.batch, c.len_t, c.table[:1])
    refused(-1, c.kv.batch, c.len_t, c.table, c.start_t[:2])
    refused(-10, c.kv.attention, 0, b, q.cpu(), out)
    refused(-5, pnb.PagedKv, 1, 4, 4, 32, 8)
    refused(-5, pnb.PagedKv, 1, 4, 4, 64, 8, page=24)
    refused(-1, pnb.PagedKv, 1, 4, 3, 64, 8)
    c.kv.attention(0, b, q, out)
    c.check(out, q)
