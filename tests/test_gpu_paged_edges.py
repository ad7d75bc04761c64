"""Calls of the paged KV cache at the ends of what its header allows, against 64 bits.

Cases, oracle and tolerances are those of the cache's other tests (test_gpu_paged.py).
"""
import math

import pytest
import torch

import transformer_decode_step_gb300 as pnb
from test_gpu_paged import DT, U, Case, _near_rotated, _rotate64, _wide

pytestmark = pytest.mark.gpu

MOST = (1 << 31) - 1


def _ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _answers(c, q, out, window):
    """Rows of tokens with entries against 64 bits; those of tokens without any are 0."""
    c.check(out, q, window)
    for b, (n, m) in enumerate(zip(c.new, c.lens)):
        dead = max(0, n - m)
        assert bool((out[c.starts[b]:c.starts[b] + dead] == 0).all())


# ----------------------------------------------------------------- windows
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window", [MOST, MOST - 1, 1 << 30, 1 << 20, 4096, 1024, 1023])
@pytest.mark.parametrize("lens,new,hd,G", [
    ([1, 0, 2, 3, 70, 1000], [4] * 6, 64, 2),           # steps: more tokens than entries
    ([1, 0, 2, 3, 70, 1000], [4] * 6, 128, 4),
    ([200, 10, 900, 0, 700], [700] * 5, 128, 4),        # several blocks, some before entry 0
    ([130, 700, 3], [700, 700, 300], 64, 1),
])
def test_windows_wider_than_the_cache(lens, new, hd, G, window, dtype):
    c = Case(lens, 2, G, hd, 32, seed=81, new=new, max_page=32)
    q = c.queries(dtype)
    out = torch.full_like(q, 7.0)
    c.kv.attention(0, c.batch(len(set(new)) > 1), q, out, window=window)
    _answers(c, q, out, window)


@pytest.mark.parametrize("window", [MOST, 1 << 30, 100])
@pytest.mark.parametrize("T", [4, 40])
def test_wide_windows_over_a_shared_prefix(T, window):
    lens = [640 + T, 900, 700, 2, 0]
    c = Case(lens, 2, 4, 64, 32, seed=82, new=[T] * 5, prefix=[([0, 1, 2], 640), ([3], 0), ([4], 0)], shared_tok=5 * T,
             max_page=_wide(5, 2, 64, 32))
    q = c.queries("fp32")
    out = torch.full_like(q, 7.0)
    c.kv.attention_shared(0, c.batch(False), _ints(0, 3, 4, 5), _ints(640, 0, 0), q, out, window=window)
    _answers(c, q, out, window)


# ------------------------------------------------- what the device's arrays hold
@pytest.mark.parametrize("n_seq", [3, 40, 700])
def test_starts_that_are_out_of_range_are_reported(n_seq):
    c = Case([20 + i % 7 for i in range(n_seq)], 2, 2, 64, 16, seed=83, new=[2] * n_seq)
    n = 2 * n_seq
    q = c.queries("fp32")
    out = torch.zeros_like(q)
    k = torch.zeros((n, 2, 64), device="cuda")
    good = c.start_t.clone()
    b = c.batch()

    def bits(at, value):
        c.start_t.copy_(good)
        if at is not None:
            c.start_t[at] = value
        c.kv.attention(0, b, q, out)
        e = c.kv.device_error()
        c.kv.append(0, b, k, k)
        assert c.kv.device_error() & ~pnb.PNB_DEV_ERR_FULL == e & ~pnb.PNB_DEV_ERR_FULL
        return e

    assert bits(None, 0) == 0
    for at in (0, 1, n_seq // 2, n_seq):
        assert bits(at, -1) == pnb.PNB_DEV_ERR_RANGE
        assert bits(at, n + 1) == pnb.PNB_DEV_ERR_RANGE
    assert bits(1, 5) == pnb.PNB_DEV_ERR_RANGE            # decreases behind it
    assert bits(n_seq, n - 3) == pnb.PNB_DEV_ERR_RANGE
    # equal starts and starts behind the first row are none
    assert bits(1, 0) == 0 and bits(0, 1) == 0 and bits(n_seq, n - 1) == 0


def test_rows_before_the_first_sequence_are_left():
    c = Case([30, 40], 2, 2, 64, 16, seed=84, new=[5, 6])
    q = c.queries("fp32", tail=4)
    c.start_t.copy_(_ints(2, 7, 13))
    b = c.batch()
    out = torch.full_like(q, 7.0)
    c.kv.attention(0, b, q, out)
    assert bool((out[:2] == 7).all()) and bool((out[13:] == 7).all())
    c.check(out[2:13], q[2:13])
    k = torch.randn((15, 2, 64), generator=c.gen, device="cuda")
    rot = torch.full_like(q, 7.0)
    before = c.kv.pages(0).clone()
    c.kv.append(0, b, k, k, q=q, q_out=rot)
    assert bool((rot[:2] == 7).all()) and bool((rot[13:] == 7).all()) and not bool((rot[2:13] == 7).any())
    e = torch.cat([torch.arange(25, 30), torch.arange(34, 40)]).cuda()
    ids = c.table.long()[torch.tensor([0] * 5 + [1] * 6, device="cuda"), e // 16]
    assert torch.equal(c.kv.pages(0)[ids, 1, :, e % 16], k[2:13].to(torch.bfloat16))
    keep = torch.ones(before.shape[0], 16, dtype=torch.bool, device="cuda")
    keep[ids, e % 16] = False
    x, y = (t.view(torch.int16).permute(0, 3, 1, 2, 4)[keep] for t in (c.kv.pages(0), before))
    assert torch.equal(x, y)
    assert c.kv.device_error() == 0


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("T", [1, 20])
def test_groups_that_are_out_of_range_are_reported(T, wide):
    c = Case([100 + T] * 4, 2, 4, 64, 16, seed=85, new=[T] * 4, prefix=[([0, 1], 64), ([2, 3], 64)], shared_tok=4 * T,
             max_page=_wide(4, 2, 64, 16) if wide else None)
    q = c.queries("fp32")
    out = torch.zeros_like(q)
    start, prefix = _ints(0, 2, 4), _ints(64, 64)
    for s, p, bad in (((0, 2, 4), (64, 64), False), ((0, 2, 4), (0, 64), False), ((0, 0, 4), (64, 0), False),
                      ((0, 2, 4), (64, -1), True), ((0, 5, 4), (64, 64), True), ((1, 2, 4), (64, 64), True),
                      ((0, 2, 3), (64, 64), True), ((0, 3, 2), (64, 64), True), ((-1, 2, 4), (64, 64), True),
                      ((0, 2, 5), (64, 64), True)):
        start.copy_(_ints(*s))
        prefix.copy_(_ints(*p))
        c.kv.attention_shared(0, c.batch(False), start, prefix, q, out)
        if bad and wide:
            assert c.kv.device_error() == pnb.PNB_DEV_ERR_RANGE, (s, p)
        else:     # (small batches do not look at groups)
            c.check(out, q)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 23])
def test_append_in_place_of_a_projection_head_by_head(n, dtype):
    # [token][head][q, k, v]: the queries' rows lie between the keys' and the values'
    hd, H = 64, 3
    c = Case([n + 5], H, 1, hd, 32, seed=86, new=[n], rope_theta=10000.0, rope_neox=True)
    x = torch.randn((n, H, 3, hd), generator=c.gen, device="cuda").to(DT[dtype])
    keep = x.clone()
    q, k, v = x.unbind(2)
    c.kv.append(0, c.batch(), k, v, q=q)
    at = torch.arange(5, n + 5, device="cuda")[None]
    _near_rotated(q, _rotate64(keep[:, :, 0], at, 10000.0, True, [hd // 2]), keep[:, :, 0], 0.0 if dtype == "fp32" else U)
    assert torch.equal(x[:, :, 1:], keep[:, :, 1:])
    e = torch.arange(5, n + 5, device="cuda")
    ids = c.table.long()[0, e // 32]
    _near_rotated(c.kv.pages(0)[ids, 0, :, e % 32], _rotate64(keep[:, :, 1], at, 10000.0, True, [hd // 2]), keep[:, :, 1], U)
    assert torch.equal(c.kv.pages(0)[ids, 1, :, e % 32], keep[:, :, 2].to(torch.bfloat16))
    for q_out in (k, v):
        with pytest.raises(pnb.PnbError) as err:
            c.kv.append(0, c.batch(), k, v, q=q, q_out=q_out)
        assert err.value.code == -1
    assert c.kv.device_error() == 0


# ------------------------------------------------ values that only some rows see
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,G,T", [(64, 4, 40), (128, 4, 40), (128, 4, 2), (64, 2, 3), (128, 1, 70)])
@pytest.mark.parametrize("value", [float("nan"), float("-inf")])
@pytest.mark.parametrize("bad", [3, 590, 660, 671])
def test_hidden_values_over_a_shared_prefix(bad, value, hd, G, T, dtype):
    # windows of 100: only the first sequences see the last of the prefix's 672 entries
    lens = [672 + T, 676 + T, 700 + T, 768 + T, 1000]
    c = Case(lens, 2, G, hd, 32, seed=87, new=[T] * 5, prefix=[(list(range(5)), 672)], shared_tok=5 * T,
             max_page=_wide(5, 2, hd, 32))
    for b in range(5):
        c.entries[b][1][bad, :, 7] = value
        c.store(b)
    q = c.queries(dtype)
    out = torch.full_like(q, 7.0)
    for window in (0, 100):
        c.kv.attention_shared(0, c.batch(False), _ints(0, 5), _ints(672), q, out, window=window)
        sees = torch.cat([(bad <= i) & ((bad > i - window) if window else torch.ones_like(i, dtype=torch.bool))
                          for i in (torch.arange(m - T, m, device="cuda") for m in lens)])
        assert not bool(torch.isfinite(out[sees][:, :, 7]).any())
        clean = Case.__new__(Case)
        clean.__dict__.update(c.__dict__)
        clean.entries = [tuple(torch.where(torch.isfinite(x), x, torch.zeros_like(x)) for x in e) for e in c.entries]
        got = out.clone()
        got[sees] = clean.want(q, window)[0][sees].to(out.dtype)
        clean.check(got, q, window)
        others = out[sees].clone()       # the value's own element is all that it reaches
        others[:, :, 7] = 0
        assert bool(torch.isfinite(others).all())


# ------------------------------------------------------------------ scores
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,T,G", [(128, 40, 4), (64, 80, 4), (64, 20, 4), (128, 90, 1), (128, 1, 4), (64, 3, 4)])
@pytest.mark.parametrize("size", [6, 8, 9, 10, 12, 16, 24, 32])
def test_answers_at_any_finite_scores(size, hd, T, G, dtype):
    # Scores of 10^size apart by as much: an entry has all of a row's weight.  Where two are near enough to be told
    # apart by less than the products' rounding (hd + 3 of 2^-24 of the sum of their sizes, in either), either may.
    c = Case([900, 333], 2, G, hd, 32, seed=88, new=[T, T])
    for negative in (False, True):
        q = c.queries(dtype, 10.0 ** size)
        if negative:      # all scores far below 0
            for b in range(2):
                c.entries[b][0].copy_(c.entries[b][0].abs())
                c.store(b)
            q = -q.abs()
        out = torch.full_like(q, 7.0)
        c.kv.attention(0, c.batch(False), q, out)
        assert bool(torch.isfinite(out).all())
        for b in range(2):
            k, v = (x.double().transpose(0, 1) for x in c.entries[b])
            rows = q[c.starts[b]:c.starts[b + 1]].double().unflatten(1, (2, G))
            s = torch.einsum("tkgd,kmd->tkgm", rows, k) / math.sqrt(hd)
            near = torch.einsum("tkgd,kmd->tkgm", rows.abs(), k.abs()) / math.sqrt(hd) * (hd + 3) * 2.0 ** -23
            m = c.lens[b]
            see = torch.arange(m, device="cuda") <= torch.arange(m - T, m, device="cuda")[:, None]
            s = s.masked_fill(~see[:, None, None], -math.inf)
            first, at = s.max(-1, keepdim=True)
            # (30: what is left of e^-30 of a weight is below every rounding)
            clear = ((s + near + 30 < first - near.gather(-1, at)).sum(-1) == m - 1)
            want = torch.gather(v[None, :, None].expand(T, -1, G, -1, -1), 3, at[..., None].expand(-1, -1, -1, 1, hd))[..., 0, :]
            got = out[c.starts[b]:c.starts[b + 1]].double().unflatten(1, (2, G))
            assert float(clear.double().mean()) > 0.5
            # the weight is off by bf16's half step, or 2^-16 with a second number, and the answer is rounded
            tol = 2.0 ** -15 if dtype == "fp32" else 2 * U
            assert float(((got - want).abs() * clear[..., None]).max()) <= tol * float(v.abs().max())
    assert c.kv.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,G,T,L", [(64, 4, 90, 300), (128, 4, 90, 300), (128, 2, 3, 700), (128, 4, 30, 5000)])
def test_rows_done_again_in_place(hd, G, T, L, dtype):
    # answers over the queries, where rows have a value that others of their tile do not see, or scores beyond any range
    c = Case([L, 40], 2, G, hd, 32, seed=89, new=[T, T], n_layer=2)
    c.kv.pages(1).copy_(c.kv.pages(0))
    q = c.queries(dtype)
    q[1::7] *= 1e12
    for b in range(2):
        c.entries[b][1][c.lens[b] - 2, :, 3] = float("nan")
        c.store(b)
    apart = torch.full_like(q, 7.0)
    c.kv.attention(0, c.batch(), q, apart)
    over = q.clone()
    c.kv.attention(0, c.batch(), over, over)
    assert torch.equal(apart.view(torch.int32 if dtype == "fp32" else torch.int16),
                       over.view(torch.int32 if dtype == "fp32" else torch.int16))
    # without the NaN, what does not attend to it is the same
    clean = torch.full_like(q, 7.0)
    c.kv.attention(1, c.batch(), q, clean)
    assert bool(torch.isfinite(clean).all())
    for b in range(2):
        rows = slice(c.starts[b], c.starts[b + 1] - 2)
        near = (apart[rows].double() - clean[rows].double()).abs()
        # (the same roundings as in test_gpu_paged.py, twice: weights' and answers')
        V = float(torch.nan_to_num(c.entries[b][1].float()).abs().max())
        calm = torch.arange(c.starts[b], c.starts[b + 1] - 2, device="cuda") % 7 != 1
        assert float(near[calm].max()) <= 2 * 2 * (2 * U if dtype == "bf16" else 2.0 ** -15) * V
        assert bool(torch.isnan(apart[c.starts[b + 1] - 2:c.starts[b + 1], :, 3]).all())
    assert c.kv.device_error() == 0
