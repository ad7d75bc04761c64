"""The paged KV cache's attention in the steady state of its kernels, against 64 bits.

A CTA takes the parts of the work that lie side by side, and small calls are spread over all of them.
These calls are large enough that a CTA goes through dozens of 128-entry tiles of one block: the
rings and the buffers of scores turn over many times, and with fp32 the sums start anew again and again.

Sequences of a case name the same pages, so that a small pool makes much work; queries are each
sequence's own.
"""
import math

import pytest
import torch

import transformer_decode_step_gb300 as pnb

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -8


class Same:
    """``B`` sequences of T tokens on the same L entries."""

    def __init__(self, L, B, T, n_kv, G, hd, page, seed, **kw):
        self.L, self.B, self.T, self.n_kv, self.G, self.H, self.hd = L, B, T, n_kv, G, n_kv * G, hd
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        n_page = -(-L // page)
        self.kv = pnb.PagedKv(n_layer=1, n_head=self.H, n_kv_head=n_kv, head_dim=hd, n_page=n_page + 1, page=page, **kw)
        self.order = torch.randperm(n_page, generator=self.gen, device="cuda")
        self.table = self.order.to(torch.int32).expand(B, -1).contiguous()
        self.lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
        self.page = page
        self.k = torch.randn((L, n_kv, hd), generator=self.gen, device="cuda").to(torch.bfloat16)
        self.v = torch.randn((L, n_kv, hd), generator=self.gen, device="cuda").to(torch.bfloat16)

    def store(self):
        pool = self.kv.pages(0)
        pool.fill_(float("nan"))
        e = torch.arange(self.L, device="cuda")
        for s, x in enumerate((self.k, self.v)):
            pool[self.order[e // self.page], s, :, e % self.page] = x
        return self.kv.batch(self.lens, self.table)

    def queries(self, dtype, scale=1.0):
        q = torch.randn((self.B * self.T, self.H, self.hd), generator=self.gen, device="cuda") * scale
        return q.to(DT[dtype])

    def want(self, q, seqs, window=0):
        """Answers of some sequences in 64 bits, [len(seqs)][T][H][hd]; the largest |score|."""
        n_kv, G, T, L = self.n_kv, self.G, self.T, self.L
        q = q.view(self.B, T, n_kv, G, self.hd)
        i = torch.arange(L - T, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")
        see = (j <= i) & ((j > i - window) if window else torch.ones_like(j <= i))
        out, most = [], 0.0
        for b in seqs:
            heads = []
            for h in range(n_kv):
                s = torch.einsum("tgd,md->tgm", q[b, :, h].double(), self.k[:, h].double()) / math.sqrt(self.hd)
                most = max(most, float(s.abs().max()))
                p = torch.softmax(s.masked_fill(~see[:, None], -math.inf), -1)
                heads.append(torch.einsum("tgm,md->tgd", p, self.v[:, h].double()))
            out.append(torch.stack(heads, 1).flatten(1, 2))
        return torch.stack(out), most


def _stairs(c, gen, chance, first, second, step):
    """Keys that move the references of the warps (32 rows of a block each) at places of their own: element w
    of a key, which rows of warp w look at, rises by ``step`` at an entry of a tile's first half (with
    ``first``) or its second one, in ``chance`` of the tiles.  Values have mean 1, so that what is
    lost of a sum shows."""
    tiles = c.L // 128
    for w in range(4):
        at = []
        for t in range(1, tiles):
            for half in ([0] if first else []) + ([1] if second else []):
                if torch.rand((), generator=gen).item() < chance:
                    at.append(t * 128 + half * 64 + int(torch.randint(0, 64, (), generator=gen)))
        rise = torch.zeros(c.L)
        rise[at] = step
        c.k[:, :, w] = torch.cumsum(rise, 0).to(torch.bfloat16).cuda()[:, None]
    c.v.copy_((c.v.float() * 0.25 + 1.0).to(torch.bfloat16))


def _looking(c, q):
    """Rows look at their warp's element of the keys, every third row at none of them."""
    q = q.view(c.B, c.T, c.n_kv, c.G, c.hd)
    q[..., :4] = 0
    row = (torch.arange(c.T)[:, None] * c.G + torch.arange(c.G)).cuda()
    for w in range(4):
        q[:, :, :, :, w] = ((row // 32 % 4 == w) & (row % 3 != 0)).to(q.dtype)[None, :, None] * math.sqrt(c.hd)
    return q.view(c.B * c.T, c.H, c.hd)


def _moving(dtype, hd, T, G, chance, first, second, B=40, window=0, L=5000):
    c = Same(L, B, T, 8, G, hd, 64, seed=5)
    gen = torch.Generator()
    gen.manual_seed(7)
    _stairs(c, gen, chance, first, second, 14.0)      # 14 of a score: 2^20 of a weight
    batch = c.store()
    q = _looking(c, c.queries(dtype))
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    c.kv.attention(0, batch, q, out, window=window)
    again = torch.empty_like(out)
    for _ in range(30):
        again.fill_(7.0)
        c.kv.attention(0, batch, q, again, window=window)
        assert torch.equal(out, again)
    assert c.kv.device_error() == 0
    seqs = list(range(0, B, 3))
    want, most = c.want(q, seqs, window)
    # Scores: at most hd / 16 * 3 additions, each cut off by 2^-23 of what it adds up, which is at most the largest
    # element (one product makes the score) and the others' random sums, below 2 * most + 64; weights: that
    # and 2^-17 (fp32) or 2^-9 (bf16); the mean's numerator and denominator: twice that, times values below 3.  Queries of
    # bf16 are exact, those of fp32 are held in 24 bits.  The output's own rounding: 2^-8 of 3 with bf16.
    score = (2 * most + 64) * (hd // 16 * 3 + 1) * 2.0 ** -23
    tol = 2 * 3 * (score + (2.0 ** -17 if dtype == "fp32" else U)) + (0 if dtype == "fp32" else U * 3)
    got = out.view(B, T, c.H, hd)[seqs].double()
    assert float((got - want).abs().max()) <= tol


# blocks of at most 128 rows: scores of the next tiles are there before the products of the last
ONE_HALF = [("fp32", 128, 32, 4), ("bf16", 128, 32, 4), ("fp32", 64, 32, 4), ("bf16", 64, 32, 4), ("fp32", 128, 64, 5)]


@pytest.mark.parametrize("dtype,hd,T,G", ONE_HALF)
@pytest.mark.parametrize("chance,first,second", [(0.3, True, True), (1.0, True, False), (1.0, False, True), (0.06, True, True)])
def test_references_that_move_beside_other_warps_products(dtype, hd, T, G, chance, first, second):
    # A warp rescales its sums in the first half of a tile while others do so in the second half of the one
    # before it or behind it; all runs answer with the same bits.  (With a step in every tile the sequences
    # are shorter, so that scores stay within what the tolerance can tell apart.)
    L = 5000 if chance < 1.0 else 2600
    _moving(dtype, hd, T, G, chance, first, second, L=L, B=40 if chance < 1.0 else 64)


@pytest.mark.parametrize("T,G,hd", [(64, 4, 64), (100, 4, 64), (37, 3, 128)])
def test_sums_that_start_anew_where_a_reference_moves(T, G, hd):
    # fp32: the reference moves in the first half of every tile, those among them that add the sums up
    _moving("fp32", hd, T, G, 1.0, True, False, L=2600, B=64)
    _moving("fp32", hd, T, G, 0.5, True, False, L=5000)


@pytest.mark.parametrize("L,T,hidden", [(400000, 64, 24), (2000000, 64, 24), (2000000, 2, 1)])
def test_a_hidden_nan_in_a_long_context_reaches_nobody_else(L, T, hidden):
    # One sequence of 304 has a NaN among its values that its first tokens do not see; the CTA that has its
    # entries has other sequences' behind them.
    B, G, hd, page = 304, 4, 64, 128
    L += 77
    c = Same(L, B, T, 1, G, hd, page, seed=9)
    batch = c.store()
    victim, bad = 150, L - T + hidden
    pool, own = c.kv.pages(0), c.kv.cfg.n_page - 1
    pool[own] = pool[c.table[0, -1].long()]
    pool[own, 1, :, bad % page, 5] = float("nan")
    assert bad // page == c.table.shape[1] - 1
    c.table[victim, -1] = own
    q = torch.randn((1, T * G, hd), generator=c.gen, device="cuda").to(torch.bfloat16).expand(B, -1, -1)
    q = q.reshape(B * T, G, hd).contiguous()
    out = torch.full_like(q, 7.0)
    c.kv.attention(0, batch, q, out)
    torch.cuda.synchronize()
    assert c.kv.device_error() == 0
    want, A = c.want(q, [0])
    # scores: 8 sums of 16 products, cut off by 2^-23 of at most twice the largest; weights by that and 2^-8 for
    # their rounding, numerator and denominator alike; answers by 2^-8 of what they are
    v = c.v
    c.v = v.abs()
    tol = 2 * (2 * A * 8 * 2.0 ** -23 + U) * float(c.want(q, [0])[0].max()) + U * float(want.abs().max())
    c.v = v
    got = out.view(B, T, G, hd).double()
    assert bool(torch.isnan(got[victim, hidden:, :, 5]).all())
    got[victim, hidden:, :, 5] = want[0, hidden:, :, 5]
    assert float((got - want).abs().max()) <= tol


@pytest.mark.parametrize("hd,T,dtype", [(64, 64, "bf16"), (128, 64, "bf16"), (64, 32, "bf16"), (128, 32, "bf16"),
                                        (64, 2, "fp32"), (128, 2, "fp32"), (64, 4, "fp32"), (128, 32, "fp32")])
def test_sums_over_a_million_entries_are_not_cut_off(hd, T, dtype):
    # All entries have the same values, so that they are the answer: the matrix units cut off what they add to a sum,
    # and with sums that go on and on answers came out 4e-3 (bf16) and 3e-4 (fp32, few rows) too small.
    c = Same(131072, 160, T, 1, 4, hd, 128, seed=3)
    c.v = (1.0 + torch.rand((1, 1, hd), generator=c.gen, device="cuda")).to(torch.bfloat16).expand_as(c.v).contiguous()
    c.store()
    table = c.table.repeat(1, 8)
    batch = c.kv.batch(torch.full((160,), 8 * c.L, dtype=torch.int32, device="cuda"), table)
    q = c.queries(dtype)
    out = torch.full_like(q, 7.0)
    c.kv.attention(0, batch, q, out)
    assert c.kv.device_error() == 0
    want = c.v[:1].double()
    if dtype == "bf16":
        # below a quarter of bf16's half step: at most 512 tiles' 8 additions at 2^-23 each, and the weights' roundings, which
        # differ from entry to entry (2^-9 / sqrt(2^20))
        assert torch.equal(out, c.v[:1].expand_as(out))
    else:
        # At most 64 additions of the matrix units between new starts are cut off by 2^-23 of a sum that is half there on
        # the average: 64 x 2^-24.  The sums of weights (2^14 additions, one per 64 entries) and of outputs (2^11) are rounded
        # either way, by at most 2^-24 of a sum that grows evenly: a deviation of 2^-24 sqrt(n / 9), taken six times for the
        # thousands of rows, 256 and 90 x 2^-24.  Weights' roundings of 2^-17, over 2^20 entries: 2^-27.
        assert float((out.double() / want - 1).abs().max()) <= (64 + 256 + 90 + 1) * 2.0 ** -24


@pytest.mark.parametrize("dtype,hd,T,L,chance", [("bf16", 64, 64, 90000, 0.02), ("bf16", 128, 64, 90000, 0.02),
                                                 ("bf16", 64, 32, 150000, 0.01), ("bf16", 128, 32, 150000, 0.01),
                                                 ("bf16", 128, 2, 20000, 0.1), ("fp32", 128, 2, 20000, 0.1),
                                                 ("fp32", 64, 4, 20000, 0.1)])
def test_references_that_move_over_long_sums(dtype, hd, T, L, chance):
    _moving(dtype, hd, T, 4, chance, True, True, L=L)


@pytest.mark.parametrize("scale", [1.0, 3.0])
@pytest.mark.parametrize("L", [300, 5000, 40000])
@pytest.mark.parametrize("hd,T,G", [(64, 64, 4), (64, 32, 4), (128, 64, 4), (128, 32, 4), (64, 4, 4), (64, 2, 4), (128, 2, 4)])
def test_precision_of_fp32(hd, T, G, L, scale):
    # Errors' rms against the answers'.  Weights are two bf16 numbers: the second holds what the first's rounding leaves, evenly
    # spread up to 2^-8, with a rounding evenly spread up to 2^-8 of that: 2^-16 / 3.  Sums of at most 64 additions, each
    # cut off by 2^-23 of a sum that is half there on the average: 32 x 2^-24 of the weighted mean, whose size they share.
    # Scores, of size `scale`: 24 additions, cut off by 2^-24 on the average (queries' 24 bits are below that).
    # All three are of random sign and independent.
    c = Same(L, 40, T, 8, G, hd, 64, seed=21)
    batch = c.store()
    q = c.queries("fp32", scale)
    seqs = [0, 17, 39]
    for qq in (q, q.to(torch.bfloat16)):
        out = torch.full(q.shape, 7.0, device="cuda")
        c.kv.attention(0, batch, qq, out)
        assert c.kv.device_error() == 0
        want, _ = c.want(qq, seqs)
        err = out.view(c.B, T, c.H, hd)[seqs].double() - want
        rel = float(err.square().mean().sqrt() / want.square().mean().sqrt())
        assert rel <= math.sqrt((2.0 ** -16 / 3) ** 2 + (32 * 2.0 ** -24) ** 2 + (24 * 2.0 ** -24 * scale) ** 2), rel
