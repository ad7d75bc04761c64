"""The 4-bit KV cache on the GPU against a plain 64-bit implementation.

Values held in the cache, ids, lengths and the eviction's choice must be equal
to the reference's.  Attention tolerances follow the kernel's roundings:

* a score x = q.k / sqrt(hd) is a sum of hd products whose fp32-side factor
  keeps 22 bits, accumulated in fp32: |dx| <= A (2^-22 + 16 * 2^-24) with
  A = sum |q_n k_n| / sqrt(hd);
* a weight's relative error is then |dx| (natural units) + 2^-21 (exponential),
  and an output, a weighted mean of values up to |v|, moves by at most twice
  the largest relative error of a weight times |v|, plus the product's own
  22-bit factor and fp32 sums (2^-20 |v|);
* a bf16 output adds its rounding (eps / 2 = 2^-8 of the value) and the single
  fp16 of its weights (2^-11 |v|).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import transformer_decode_step_gb300 as pnb  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


def held(x):
    """What the cache stands for after storing rows x [..., hd], in 64 bits."""
    x = x.detach().double().cpu().numpy()
    b = x.reshape(x.shape[:-1] + (-1, 32))
    top = np.abs(b).max(-1, keepdims=True)
    with np.errstate(over="ignore", invalid="ignore"):
        d = np.minimum(top / 7.0, 65504.0).astype(np.float16).astype(np.float64)
        u = np.clip(np.rint(b / np.where(d == 0, 1.0, d)), -8, 7)
    y = u * d
    y[~np.isfinite(top[..., 0])] = np.nan
    return torch.from_numpy(y.reshape(x.shape)).cuda()


class Ref:
    """A plain cache: per slot and KV head the held rows, ids and weights (64 bits)."""

    def __init__(self, n_slot, n_head, n_kv, hd, cap):
        self.B, self.H, self.Hkv, self.hd, self.cap = n_slot, n_head, n_kv, hd, cap
        z = lambda *s: torch.zeros(s, dtype=torch.float64, device="cuda")
        self.k, self.v = z(n_slot, n_kv, cap, hd), z(n_slot, n_kv, cap, hd)
        self.w = z(n_slot, n_kv, cap)
        self.ids = torch.zeros((n_slot, n_kv, cap), dtype=torch.int64, device="cuda")
        self.len, self.seen = [0] * n_slot, [0] * n_slot

    def append(self, k, v, n_new=None, start=None):
        hk, hv = held(k), held(v)
        for b in range(self.B):
            n = k.shape[1] if n_new is None else n_new[b]
            s = self.len[b] if start is None else start[b]
            seen = self.seen[b] - (self.len[b] - s)
            n = min(n, self.cap - s)
            self.k[b, :, s:s + n] = hk[b, :n].transpose(0, 1)
            self.v[b, :, s:s + n] = hv[b, :n].transpose(0, 1)
            self.w[b, :, s:s + n] = 0
            self.ids[b, :, s:s + n] = torch.arange(seen, seen + n, device="cuda")
            self.len[b], self.seen[b] = s + n, seen + n

    def attention(self, q, decay=None):
        """(output, tolerance without the output type's, weights' tolerance)"""
        B, T, H, hd = q.shape
        G = H // self.Hkv
        out = torch.zeros((B, T, H, hd), dtype=torch.float64, device="cuda")
        tol = torch.zeros((B, T, H, 1), dtype=torch.float64, device="cuda")
        wtol = 0.0
        new = torch.zeros_like(self.w)
        for b in range(B):
            for t in range(T):
                m = self.len[b] - T + 1 + t
                if m <= 0:
                    continue
                qq = q[b, t].double().reshape(self.Hkv, G, hd)
                k, v = self.k[b, :, :m], self.v[b, :, :m]
                x = torch.einsum("hgd,hnd->hgn", qq, k) / hd ** 0.5
                p = torch.softmax(x, -1)
                out[b, t] = torch.einsum("hgn,hnd->hgd", p, v).reshape(H, hd)
                new[b, :, :m] += p.sum(1)
                a = torch.einsum("hgd,hnd->hgn", qq.abs(), k.abs()).amax(-1) / hd ** 0.5
                rel = a * (2.0 ** -22 + 16 * 2.0 ** -24) + 2.0 ** -21
                big = v.abs().amax((1, 2))[:, None]
                tol[b, t] = ((2 * rel + 2.0 ** -20) * big).reshape(H, 1)
                wtol = max(wtol, float(2 * rel.max()) * G * T)
        if decay is not None:
            for b in range(B):
                n = self.len[b]
                self.w[b, :, :n] = decay * self.w[b, :, :n] + new[b, :, :n] if decay else new[b, :, :n]
        return out, tol, wtol

    def evict(self, budget, n_sink=0, n_recent=0, w=None):
        """The new arrangement; w: the weights to choose by (the kernel's own fp32 ones)."""
        w = self.w if w is None else w
        for b in range(self.B):
            n = self.len[b]
            if n <= budget:
                continue
            for h in range(self.Hkv):
                ids = self.ids[b, h, :n].cpu().numpy()
                wt = w[b, h, :n].double().cpu().numpy()
                stay = (ids < n_sink) | (ids >= self.seen[b] - n_recent)
                rest = np.flatnonzero(~stay)
                rest = rest[np.argsort(-wt[rest], kind="stable")][:budget - int(stay.sum())]
                stay[rest] = True
                src = np.arange(budget)
                src[~stay[:budget]] = budget + np.flatnonzero(stay[budget:])
                s = torch.from_numpy(src).cuda()
                for a in (self.k, self.v, self.w, self.ids):
                    a[b, h, :budget] = a[b, h, s]
            self.len[b] = budget


def make(n_slot, n_head, n_kv, hd, cap, n_layer=1, track=0):
    """A cache whose buffer starts full of NaN scales and wild codes."""
    c = pnb.Kv4Cache(n_layer, n_slot, n_head, n_kv, hd, cap, track=track)
    c.buf.fill_(0xFF)
    c.reset()
    return c


def rows(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check_content(c, ref, layer=0):
    B, n = ref.B, max(ref.len + [1])
    k = torch.full((B, n, ref.Hkv, ref.hd), 7.0, device="cuda")
    v = torch.full_like(k, 7.0)
    c.read(layer, k, v)
    assert c.lengths(layer).tolist() == ref.len
    assert c.seen(layer).tolist() == ref.seen
    for b in range(B):
        m = ref.len[b]
        for got, want in ((k, ref.k), (v, ref.v)):
            w = want[b, :, :m].transpose(0, 1)
            g = got[b, :m].double()
            assert torch.equal(torch.isnan(g), torch.isnan(w))
            assert torch.equal(torch.nan_to_num(g), torch.nan_to_num(w))
            assert not got[b, m:].any()
        assert torch.equal(c.ids(layer)[b, :, :m].long(), ref.ids[b, :, :m])


def check_attention(c, ref, q, out_dtype=None, decay=None, layer=0):
    out = torch.full(q.shape, float("nan"), dtype=out_dtype or q.dtype, device="cuda")
    c.attention(layer, q, out, decay=decay)
    want, tol, wtol = ref.attention(q, decay)
    if out.dtype == BF16:
        tol = tol + want.abs() * 2.0 ** -8 + tol_fp16(ref)
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), f"max error {float((err - tol).max()):.3e} over tolerance"
    if decay is not None:
        w = c.weights(layer)
        for b in range(ref.B):
            n = ref.len[b]
            d = (w[b, :, :n].double() - ref.w[b, :, :n]).abs()
            assert n == 0 or float(d.max()) <= wtol + 2.0 ** -22 * float(ref.w[b, :, :n].max())
    return out


def tol_fp16(ref):
    """A bf16 output's weights are single fp16 numbers: 2^-11 of the largest value."""
    big = max(float(ref.v[b, :, :n].abs().max()) for b, n in enumerate(ref.len) if n) if any(ref.len) else 0.0
    return 2.0 ** -11 * big


# ------------------------------------------------------------ append / read
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 31, 33, 100])
def test_append_holds_the_definition(hd, dtype, T):
    c, ref = make(3, 6, 3, hd, 128), Ref(3, 6, 3, hd, 128)
    k, v = rows((3, T, 3, hd), 1, dtype, 3.0), rows((3, T, 3, hd), 2, dtype, 0.1)
    n = [T, 0, (T + 1) // 2]
    c.append(0, k, v, n_new=i32(n))
    ref.append(k, v, n)
    check_content(c, ref)
    assert c.device_error() == 0


def test_append_piecewise_equals_at_once():
    k, v = rows((2, 95, 2, 64), 3, BF16), rows((2, 95, 2, 64), 4, BF16)
    whole = make(2, 2, 2, 64, 96)
    whole.append(0, k, v)
    c = make(2, 2, 2, 64, 96)
    at = 0
    for n in (1, 2, 5, 24, 31, 1, 31):
        c.append(0, k[:, at:at + n], v[:, at:at + n])
        at += n
    assert at == 95
    a, b = torch.empty(2, 2, 95, 2, 64, device="cuda"), torch.empty(2, 2, 95, 2, 64, device="cuda")
    whole.read(0, a[0], a[1])
    c.read(0, b[0], b[1])
    assert torch.equal(a, b)
    assert torch.equal(whole.ids(0)[..., :95], c.ids(0)[..., :95])


def test_quantiser_borders():
    """Quotients exactly between two codes, subnormal scales, zero, huge and non-finite rows."""
    hd = 32
    x = torch.zeros(1, 9, 1, hd, dtype=torch.float64)
    d = 0.3017578125                                     # an fp16 number
    x[0, 0, 0, :16] = (torch.arange(16) - 7.5) * d       # ties, the largest beyond 7 d
    x[0, 0, 0, 16] = 7 * d
    x[0, 0, 0, :16] = x[0, 0, 0, :16].clamp(-7 * d, 7 * d)
    x[0, 1, 0] = torch.linspace(-1, 1, hd) * 7 * 2.0 ** -24 * 1.4   # scale rounds to a subnormal
    x[0, 2, 0] = torch.linspace(-1, 1, hd) * 2.0 ** -26  # scale rounds to zero
    x[0, 4, 0, 3] = 1e30                                 # scale saturates
    x[0, 5, 0, 5] = float("nan")
    x[0, 6, 0, 5] = float("inf")
    x[0, 7, 0, 5] = -float("inf")
    x[0, 8, 0, 0] = -1.0                                 # one negative entry: u = 8 - 7
    x = x.float().cuda()
    # ties a half ulp away in either direction are no ties
    y = x.clone()
    y[0, 0, 0, 1] = torch.nextafter(y[0, 0, 0, 1], torch.tensor(0.0, device="cuda"))
    y[0, 0, 0, 2] = torch.nextafter(y[0, 0, 0, 2], torch.tensor(-9.0, device="cuda"))
    c, ref = make(1, 1, 1, hd, 32), Ref(1, 1, 1, hd, 32)
    c.append(0, x, y)
    ref.append(x, y)
    check_content(c, ref)


def test_quantiser_many_values():
    """Every quotient of 2^21 fp32 values, many of them near a border."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    n = 1 << 9
    top = torch.rand((1, n, 32, 4, 1), generator=g, device="cuda") * 4 + 0.01
    d = (top / torch.full_like(top, 7.0)).half().float()
    steps = torch.randint(-13, 14, (1, n, 32, 4, 32), generator=g, device="cuda").float() * 0.5
    x = steps * d
    x = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.5, x,
                    torch.nextafter(x, x * 2))
    x[..., :1] = top
    x = torch.minimum(x, top).reshape(1, n, 32, 128)
    c, ref = make(1, 32, 32, 128, n), Ref(1, 32, 32, 128, n)
    c.append(0, x, -x)
    ref.append(x, -x)
    check_content(c, ref)


@pytest.mark.parametrize("hd", [32, 128])
def test_quantiser_bf16_ties(hd):
    """bf16 quotients that are half an integer exactly (scales that are powers of two and seven
    times them), and every bf16 magnitude against a fixed scale."""
    n = 1 << 10
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    e = torch.randint(-12, 9, (1, n, 2, hd // 32, 1), generator=g, device="cuda").float()
    d = torch.exp2(e) * torch.where(torch.rand(e.shape, generator=g, device="cuda") < 0.5, 1.0, 1.25)
    x = torch.randint(-13, 14, (1, n, 2, hd // 32, 32), generator=g, device="cuda").float() * 0.5 * d
    x[..., 0:1] = 7 * d
    ties = x.to(BF16)
    assert torch.equal(ties.float(), x)      # halves of the scale are bf16 numbers
    # magnitudes from 2^-32 up to 7, all bf16 numbers among them, in blocks whose largest is 7
    every = torch.arange(0x2f80, 0x40e0, dtype=torch.int16, device="cuda").view(BF16)
    blocks = n * 2 * (hd // 32)
    y = torch.full((blocks, 32), 7.0, dtype=BF16, device="cuda")
    at = torch.arange(blocks * 31, device="cuda") % every.numel()
    y[:, 1:] = every[at].view(blocks, 31)
    c, ref = make(1, 2, 2, hd, n), Ref(1, 2, 2, hd, n)
    v = y.reshape(1, n, 2, hd)
    c.append(0, ties.reshape(1, n, 2, hd), v)
    ref.append(ties.reshape(1, n, 2, hd), v)
    check_content(c, ref)
    c.reset()
    c.append(0, -v, v * -0.5)                # the other sign, and a scale of one half
    ref = Ref(1, 2, 2, hd, n)
    ref.append(-v, v * -0.5)
    check_content(c, ref)


@pytest.mark.parametrize("T", [64, 96])      # the one-CTA-per-slot form and the chunked one
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hard", [False, True])
def test_quantiser_quotient_of_seven_and_a_half(T, dtype, hard):
    """Blocks whose largest magnitude is 7.5 d exactly (d subnormal: n 2^-24, n = 1..6, the fp16 number
    next to 7.5 n 2^-24 / 7): +7.5 rounds to the even 8 and is held as 7, at each place of a code
    word, whatever other blocks (``hard``: a quotient above 7.5) share the warp."""
    n = torch.arange(T) % 6 + 1
    sign, at = 1.0 - 2.0 * (torch.arange(T) // 6 % 2), torch.arange(T) // 6 % 8
    g = torch.Generator()
    g.manual_seed(360)
    d = n[:, None] * 2.0 ** -24
    x = torch.randint(-6, 7, (T, 32), generator=g) * d
    x[torch.arange(T), at + 8 * (torch.arange(T) % 4)] = 7.5 * sign * d[:, 0]
    other = torch.randint(-6, 7, (T, 32), generator=g) * d
    if hard:
        other = torch.where(torch.arange(32) % 5 == 0, 8 * 2.0 ** -24, other.clamp(-6 * 2.0 ** -24, 6 * 2.0 ** -24))
    x, other = (t.view(1, T, 1, 32).cuda().to(dtype) for t in (x, other))
    assert float(x.double().abs().max()) == 45 * 2.0 ** -24 and not torch.equal(x, other)
    assert torch.equal(held(x).abs().amax(-1)[0, :, 0].cpu(), (7.0 + (sign < 0)) * d[:, 0].double())
    c = make(1, 1, 1, 32, 96)
    for k, v in ((x, other), (other, x)):
        c.reset()
        ref = Ref(1, 1, 1, 32, 96)
        c.append(0, k, v)
        ref.append(k, v)
        check_content(c, ref)


@pytest.mark.parametrize("n_slot,n_kv,hd,T", [(3, 2, 128, 8), (300, 4, 128, 8), (300, 4, 128, 3), (5, 40, 32, 2),
                                              (2, 1, 64, 16), (2, 1, 64, 17), (1, 64, 128, 1), (4, 3, 128, 9)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_append_and_read_forms(n_slot, n_kv, hd, T, dtype):
    """The one-CTA-per-slot and the chunked forms, from starts inside and at the ends of chunks, with
    neighbouring entries kept, and reads that begin inside, at and behind a slot's end."""
    cap = 96
    c, ref = make(n_slot, n_kv, n_kv, hd, cap), Ref(n_slot, n_kv, n_kv, hd, cap)
    lens = [(29 + 13 * b) % 64 for b in range(n_slot)]
    k, v = rows((n_slot, 64, n_kv, hd), 300, dtype), rows((n_slot, 64, n_kv, hd), 301, dtype)
    c.append(0, k, v, n_new=i32(lens))
    ref.append(k, v, lens)
    n = [T - b % 2 for b in range(n_slot)]
    start = [max(0, m - b % 4) for b, m in enumerate(lens)]
    k, v = rows((n_slot, T, n_kv, hd), 302, dtype), rows((n_slot, T, n_kv, hd), 303, dtype)
    c.append(0, k, v, n_new=i32(n), start=i32(start))
    ref.append(k, v, n, start)
    check_content(c, ref)
    assert c.device_error() == 0
    first = [(m + b % 3 - 1) if b % 5 else (-1, cap, cap + 40, 1 << 30)[b // 5 % 4] for b, m in enumerate(start)]
    yk, yv = torch.full_like(k, 9.0), torch.full_like(v, 9.0)
    c.read(0, yk, yv, first=i32(first))
    for b, f in enumerate(first):
        for got, want in ((yk, ref.k), (yv, ref.v)):
            w = torch.zeros((T, n_kv, hd), dtype=torch.float64, device="cuda")
            m = min(T, ref.len[b] - f) if f >= 0 else 0
            if m > 0:
                w[:m] = want[b, :, f:f + m].transpose(0, 1)
            assert torch.equal(got[b], w.to(dtype))


def test_append_reads_strided_rows():
    """K and V inside a fused QKV projection, and in a state's [head][position][hd] cache layout."""
    B, T, H, Hkv, hd = 2, 9, 4, 2, 64
    fused = rows((B, T, (H + 2 * Hkv) * hd), 6, BF16)
    k = fused[..., H * hd:(H + Hkv) * hd].view(B, T, Hkv, hd)
    v = fused[..., (H + Hkv) * hd:].view(B, T, Hkv, hd)
    c, ref = make(B, H, Hkv, hd, 64), Ref(B, H, Hkv, hd, 64)
    c.append(0, k, v)
    ref.append(k, v)
    cache = rows((2, B, Hkv, 40, hd), 7)
    k, v = cache[0].transpose(1, 2), cache[1].transpose(1, 2)
    c.append(0, k, v, n_new=i32([40, 17]))
    ref.append(k, v, [40, 17])
    check_content(c, ref)
    # and read back into that layout, rounded to bf16
    back = torch.zeros((2, B, Hkv, 50, hd), dtype=BF16, device="cuda")
    c.read(0, back[0].transpose(1, 2)[:, :30], back[1].transpose(1, 2)[:, :30], first=i32([4, 19]))
    for b, f in enumerate((4, 19)):
        n = min(30, ref.len[b] - f)
        assert torch.equal(back[0, b, :, :n], ref.k[b, :, f:f + n].to(BF16))
        assert torch.equal(back[1, b, :, :n], ref.v[b, :, f:f + n].to(BF16))
        assert not back[:, b, :, n:].any()


def test_rollback_and_capacity():
    c, ref = make(2, 2, 1, 32, 64), Ref(2, 2, 1, 32, 64)
    k, v = rows((2, 60, 1, 32), 8), rows((2, 60, 1, 32), 9)
    c.append(0, k, v)
    ref.append(k, v)
    k2, v2 = rows((2, 5, 1, 32), 10), rows((2, 5, 1, 32), 11)
    c.append(0, k2, v2, n_new=i32([5, 3]), start=i32([57, 60]))   # slot 0 takes back 3 drafts
    ref.append(k2, v2, [5, 3], [57, 60])
    check_content(c, ref)
    assert c.device_error() == 0
    c.append(0, k2, v2)                       # 62 + 5 and 63 + 5 pass the capacity
    ref.append(k2, v2)
    check_content(c, ref)
    assert ref.len == [64, 64] and c.device_error() == pnb.PNB_DEV_ERR_FULL
    c.reset()
    assert c.device_error() == 0 and c.lengths(0).tolist() == [0, 0]
    # starts and counts out of range leave the slot alone
    c.append(0, k2, v2, start=i32([1, 0]))
    assert c.lengths(0).tolist() == [0, 5] and c.device_error() == pnb.PNB_DEV_ERR_RANGE
    c.append(0, k2, v2, n_new=i32([6, -1]))
    assert c.lengths(0).tolist() == [0, 5] and c.seen(0).tolist() == [0, 5]


def test_reset_of_one_slot_and_layers():
    c = make(2, 2, 2, 32, 32, n_layer=2)
    k = rows((2, 3, 2, 32), 12)
    for layer in (0, 1):
        c.append(layer, k, k)
    c.append(1, k, k)
    assert c.lengths(0).tolist() == [3, 3] and c.lengths(1).tolist() == [6, 6]
    c.reset(1)
    assert c.lengths(0).tolist() == [3, 0] and c.lengths(1).tolist() == [6, 0]


# --------------------------------------------------------------- attention
SHAPES = [  # n_kv, group, head_dim, T
    (2, 1, 128, 1), (2, 4, 128, 1), (1, 8, 128, 1), (3, 3, 64, 1), (2, 7, 32, 1), (1, 16, 64, 1),
    (2, 4, 128, 3), (4, 1, 64, 9), (1, 5, 32, 8), (1, 64, 128, 1), (1, 1, 32, 64),
]


@pytest.mark.parametrize("n_kv,G,hd,T", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_against_64_bits(n_kv, G, hd, T, dtype):
    lens = [0, 1, 2, 31, 32, 33, 64, 65, 200, 257]
    B, cap = len(lens), 288
    c, ref = make(B, n_kv * G, n_kv, hd, cap), Ref(B, n_kv * G, n_kv, hd, cap)
    k, v = rows((B, max(lens), n_kv, hd), 13, BF16, 2.0), rows((B, max(lens), n_kv, hd), 14, BF16)
    c.append(0, k, v, n_new=i32(lens))
    ref.append(k, v, lens)
    check_attention(c, ref, rows((B, T, n_kv * G, hd), 15, dtype, 2.0))
    assert c.device_error() == 0


@pytest.mark.parametrize("q_dtype,out_dtype", [(F32, BF16), (BF16, F32)])
def test_attention_types_may_differ(q_dtype, out_dtype):
    c, ref = make(2, 4, 2, 64, 96), Ref(2, 4, 2, 64, 96)
    k, v = rows((2, 90, 2, 64), 16), rows((2, 90, 2, 64), 17)
    c.append(0, k, v, n_new=i32([90, 41]))
    ref.append(k, v, [90, 41])
    check_attention(c, ref, rows((2, 1, 4, 64), 18, q_dtype), out_dtype)


@pytest.mark.parametrize("hd,n_kv,G,B,n", [(128, 1, 8, 1, 20011), (128, 8, 4, 2, 5003), (64, 2, 4, 1, 9001),
                                           (32, 1, 1, 1, 40961), (128, 2, 1, 300, 70)])
def test_attention_split_over_many_ctas(hd, n_kv, G, B, n):
    cap = -(-n // 32) * 32
    c, ref = make(B, n_kv * G, n_kv, hd, cap, track=1), Ref(B, n_kv * G, n_kv, hd, cap)
    lens = [max(1, n - 17 * b) if B < 10 else 1 + (37 * b) % n for b in range(B)]
    k, v = rows((B, n, n_kv, hd), 19, BF16, 1.5), rows((B, n, n_kv, hd), 20, BF16)
    c.append(0, k, v, n_new=i32(lens))
    ref.append(k, v, lens)
    q = rows((B, 1, n_kv * G, hd), 21, F32, 2.0)
    a = check_attention(c, ref, q, decay=0.0)
    w = c.weights(0).clone()
    for _ in range(3):                        # the same call gives the same bits
        b = torch.empty_like(a)
        c.attention(0, q, b, decay=0.0)
        assert torch.equal(a, b)
        for i, m in enumerate(lens):
            assert torch.equal(w[i, :, :m], c.weights(0)[i, :, :m])


@pytest.mark.parametrize("B,n_kv,G,hd,lo,hi", [
    (1024, 1, 1, 32, 0, 40),       # the most slots
    (1024, 2, 4, 128, 5, 5),       # more items than CTAs, all alike
    (3, 4, 2, 128, 99, 99),        # items of equal, short length: a CTA each
    (5, 3, 8, 64, 1, 300),         # ragged and short
    (2, 64, 1, 128, 700, 1000),
])
def test_attention_work_splits(B, n_kv, G, hd, lo, hi):
    cap = -(-hi // 32) * 32
    c, ref = make(B, n_kv * G, n_kv, hd, cap, track=1), Ref(B, n_kv * G, n_kv, hd, cap)
    lens = [lo + (37 * b) % (hi - lo + 1) for b in range(B)]
    k, v = rows((B, hi, n_kv, hd), 310, BF16, 1.5), rows((B, hi, n_kv, hd), 311, BF16)
    c.append(0, k, v, n_new=i32(lens))
    ref.append(k, v, lens)
    for dtype in (F32, BF16):
        check_attention(c, ref, rows((B, 1, n_kv * G, hd), 312, dtype, 2.0), decay=0.0)
    assert c.device_error() == 0


@pytest.mark.parametrize("longest", [31, 832, 833])      # below, at and past what one CTA keeps whole
@pytest.mark.parametrize("B,n_kv,G,hd,T", [(2, 3, 2, 128, 1), (37, 4, 8, 64, 3), (70, 3, 1, 128, 2), (9, 32, 4, 32, 5)])
def test_attention_ragged_slots_some_empty(B, n_kv, G, hd, T, longest):
    c, ref = make(B, n_kv * G, n_kv, hd, 864, track=T), Ref(B, n_kv * G, n_kv, hd, 864)
    lens = [longest if b == B // 2 else 0 if b % 5 == 4 else (53 * b * b) % (longest + 1) for b in range(B)]
    k, v = rows((B, longest, n_kv, hd), 313, BF16, 1.5), rows((B, longest, n_kv, hd), 314, BF16)
    c.append(0, k, v, n_new=i32(lens))
    ref.append(k, v, lens)
    q = rows((B, T, n_kv * G, hd), 315, F32, 2.0)
    a = check_attention(c, ref, q, decay=0.0)
    check_attention(c, ref, q.to(BF16))
    b = torch.empty_like(a)
    c.attention(0, q, b)
    assert torch.equal(a, b)                  # the same bits, tracked or not
    assert c.device_error() == 0


def test_offsets_past_32_bits():
    """A cache of 10 GB and 2^32 tracked scores: the last slot's entries, scores and moves lie behind
    4 GiB.  Rows of all slots are one tensor's (slot stride 0); the other slots stay empty."""
    B, n_kv, G, hd, T, cap = 64, 8, 8, 128, 8, 1 << 17
    n = cap - 5
    c = make(B, n_kv * G, n_kv, hd, cap, track=T)
    assert c.buf.numel() > 9 << 30 and B * n_kv * G * T * cap >= 1 << 32
    k, v = rows((1, n, n_kv, hd), 340, BF16), rows((1, n, n_kv, hd), 341, BF16)
    c.append(0, k.expand(B, n, n_kv, hd), v.expand(B, n, n_kv, hd), n_new=i32([0] * (B - 1) + [n]))
    q = rows((B, T, n_kv * G, hd), 342, BF16, 2.0)
    out = torch.empty((B, T, n_kv * G, hd), device="cuda")
    c.attention(0, q, out, decay=0.0)
    assert not out[:-1].any() and c.device_error() == 0
    ref = Ref(1, n_kv * G, n_kv, hd, cap)     # the last slot alone
    ref.append(k, v)
    want, tol, wtol = ref.attention(q[-1:], 0.0)
    assert bool(((out[-1:].double() - want).abs() <= tol).all())
    w = c.weights(0)[-1]
    assert float((w[:, :n].double() - ref.w[0, :, :n]).abs().max()) <= wtol
    ref.w[0].copy_(w.double())
    c.evict(0, 60000, 4, 100)
    ref.evict(60000, 4, 100)
    assert c.lengths(0).tolist() == [0] * (B - 1) + [60000]
    assert torch.equal(c.ids(0)[-1, :, :60000].long(), ref.ids[0, :, :60000])
    first = i32([0] * (B - 1) + [59990])
    yk = torch.empty((B, 20, n_kv, hd), device="cuda")
    yv = torch.empty_like(yk)
    c.read(0, yk, yv, first=first)
    for got, held_rows in ((yk, ref.k), (yv, ref.v)):
        assert torch.equal(got[-1, :10].double(), held_rows[0, :, 59990:60000].transpose(0, 1))
        assert not got[-1, 10:].any() and not got[:-1].any()


def test_extreme_values():
    """A score far above the others late in the sequence, V scales that grow by 2^20 along it
    (the fp16 products' reference moves), large and tiny queries."""
    B, n, hd = 4, 400, 64
    k, v = rows((B, n, 1, hd), 22), rows((B, n, 1, hd), 23)
    v = v * torch.logspace(-4, 2, n, device="cuda")[None, :, None, None]
    k[1, 350] *= 40
    q = rows((B, 1, 2, hd), 24)
    q[2] *= 1e-20
    q[3] *= 30
    c, ref = make(B, 2, 1, hd, 416), Ref(B, 2, 1, hd, 416)
    c.append(0, k, v)
    ref.append(k, v)
    check_attention(c, ref, q)
    # values that shrink instead, and rows of zeros
    v = v.flip(1).contiguous()
    v[0, 100:] = 0
    c.reset()
    ref = Ref(B, 2, 1, hd, 416)
    c.append(0, k, v)
    ref.append(k, v)
    check_attention(c, ref, q)


@pytest.mark.parametrize("exponent", [20, 27, 28, 31, 60, 106, 119, 123])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n_kv,G,T,n", [(2, 1, 1, 300), (1, 4, 2, 300), (2, 2, 1, 5000)])
def test_attention_at_very_large_scores(n_kv, G, T, n, dtype, exponent):
    """Queries up to 2^124 along one dim in which the keys hold whole numbers c <= 7: the scores of
    the largest c lie above all others by far more than 100, so the answer is the mean of those entries'
    values and they share the weight.  fp32 sums of equal terms: 2^-20 of the values covers them."""
    B, hd = 3, 64
    cap = -(-n // 32) * 32
    g = torch.Generator(device="cuda")
    g.manual_seed(370)
    c = torch.randint(-7, 7, (B, n, n_kv), generator=g, device="cuda")
    c[torch.rand((B, n, n_kv), generator=g, device="cuda") < 0.02] = 7
    c[:, 0] = 7                                   # every query token sees it
    k = torch.zeros((B, n, n_kv, hd), device="cuda")
    k[..., 5] = c
    k[..., 6] = 7                                 # the block's scale is 1
    v = rows((B, n, n_kv, hd), 371)
    q = torch.zeros((B, T, n_kv * G, hd), device="cuda")
    q[..., 5] = (1 + torch.rand(q.shape[:3], generator=g, device="cuda")) * 2.0 ** exponent
    q = q.to(dtype)
    cache, ref = make(B, n_kv * G, n_kv, hd, cap, track=T), Ref(B, n_kv * G, n_kv, hd, cap)
    cache.append(0, k, v)
    ref.append(k, v)
    assert torch.equal(ref.k[:, :, :n, 5], c.permute(0, 2, 1).double())
    out = torch.empty_like(q)
    cache.attention(0, q, out, decay=0.0)
    weights = torch.zeros((B, n_kv, n), dtype=torch.float64, device="cuda")
    for t in range(T):
        m = n - T + 1 + t
        p = (c[:, :m] == 7).permute(0, 2, 1).double()
        p /= p.sum(-1, keepdim=True)
        weights[..., :m] += G * p
        want = torch.einsum("bhn,bhnd->bhd", p, ref.v[:, :, :m]).repeat_interleave(G, 1)
        tol = 2.0 ** -20 * ref.v.abs().max() + (0 if dtype == F32 else 2.0 ** -8 * want.abs() + 2.0 ** -11 * ref.v.abs().max())
        assert bool(((out[:, t].double() - want).abs() <= tol).all())
    # roundings of an exponential (2^-22), a sum, its reciprocal and a product, over G T rows
    assert bool(((cache.weights(0)[..., :n].double() - weights).abs() <= 2.0 ** -19 * weights + 1e-30).all())


def plain_fp32(ref, q):
    """Outputs and weights of a plain fp32 computation on the held values, and the largest score."""
    B, T, H, hd = q.shape
    n, G = max(ref.len), H // ref.Hkv
    kk, vv = ref.k[:, :, :n].float(), ref.v[:, :, :n].float()
    qq = q.float().view(B, T, ref.Hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, ref.Hkv, T * G, hd)
    x = torch.matmul(qq, kk.transpose(2, 3)) * hd ** -0.5
    limit = torch.arange(n - T + 1, n + 1, device="cuda").repeat_interleave(G)[:, None]
    p = torch.softmax(torch.where(torch.arange(n, device="cuda") < limit, x, -torch.inf), -1)
    out = torch.matmul(p, vv).view(B, ref.Hkv, T, G, hd).permute(0, 2, 1, 3, 4).reshape(B, T, H, hd)
    return out, p.sum(2), float(x.abs().max())


def check_as_exact_as_plain(c, ref, q):
    """The fp32 output's error, in the norm over each 32-dim block, is at most twice that of plain fp32
    (both are random sums over the rows and entries), plus one rounding, plus what is not random: an entry
    that holds most of a row's weight moves the whole row by its score's error.  A score x of this cache is
    rounded where its halves' sums meet (2^-24 of it, 2^-23 if cut off), by its block's scale and by the
    softmax's scale (2^-24 each), 4 * 2^-24 |x| in all; plain fp32 has one or two of these."""
    out = torch.empty(q.shape, device="cuda")
    c.attention(0, q, out, decay=0.0)
    want = ref.attention(q, 0.0)[0]
    plain, pw, top = plain_fp32(ref, q)
    one = 2.0 ** -23 + 4 * 2.0 ** -24 * top
    norm = lambda a: a.double().unflatten(-1, (-1, 32)).transpose(-1, -2).reshape(-1, a.shape[-1] // 32).norm(dim=0)
    assert bool((norm(out - want) <= 2 * norm(plain - want) + one * norm(want)).all()), \
        (norm(out - want) / norm(want), norm(plain - want) / norm(want))
    n = max(ref.len)
    w, err = ref.w[:, :, :n], lambda a: float((a.double() - ref.w[:, :, :n]).norm())
    assert err(c.weights(0)[:, :, :n]) <= 2 * err(pw) + one * float(w.norm())


@pytest.mark.parametrize("n_kv,G,hd,T", [(4, 1, 64, 1), (2, 4, 128, 1), (1, 8, 32, 1), (1, 4, 128, 3)])
@pytest.mark.parametrize("n", [60, 2304, 20000])
@pytest.mark.parametrize("above,size", [(0.0, 0.4), (4.0, 0.4), (6.0, 0.08), (8.0, 1e-3), (8.0, 30.0)])
def test_attention_beside_a_sink(n_kv, G, hd, T, n, above, size):
    """The first entry's value is 0 and it holds 1 - e^-above of the weight or more (above 0: about half);
    the others' small shares make the output."""
    B = 4
    cap = -(-n // 32) * 32
    k, v = rows((B, n, n_kv, hd), 380), rows((B, n, n_kv, hd), 381, F32, size)
    q = rows((B, T, n_kv * G, hd), 382)
    q[..., 0] = 4.0
    k[..., 0] = 0
    k[:, 0] = 0
    k[:, 0, :, 0] = (np.log(n) + 0.5 + above) * hd ** 0.5 / 4
    v[:, 0] = 0
    c, ref = make(B, n_kv * G, n_kv, hd, cap, track=T), Ref(B, n_kv * G, n_kv, hd, cap)
    c.append(0, k, v)
    ref.append(k, v)
    check_as_exact_as_plain(c, ref, q)
    ref.attention(q, 0.0)
    share = ref.w[:, :, 0] / (T * G)
    assert bool((share > 1 - 4 * np.exp(-above)).all()) and (above or 0.2 < float(share.mean()) < 0.8)


@pytest.mark.parametrize("G", [1, 8])
def test_attention_values_of_unlike_size(G):
    """A block of 32 dims whose values are 100 times the others', single entries whose values are, and
    scores spread so that far entries weigh 2^-20 of near ones."""
    B, n, n_kv, hd = 4, 3000, 2, 128
    k, v = rows((B, n, n_kv, hd), 383), rows((B, n, n_kv, hd), 384, F32, 0.05)
    q = rows((B, 1, n_kv * G, hd), 385)
    v[0, :, :, 32:64] *= 100
    v[1, ::97] *= 100
    q[..., 0] = 4.0
    k[2:, :, :, 0] = torch.linspace(-14, 0, n, device="cuda")[:, None] * hd ** 0.5 / 4
    k[3] = k[3].flip(0)
    c, ref = make(B, n_kv * G, n_kv, hd, 3008, track=1), Ref(B, n_kv * G, n_kv, hd, 3008)
    c.append(0, k, v)
    ref.append(k, v)
    check_as_exact_as_plain(c, ref, q)


@pytest.mark.parametrize("G", [1, 8])
def test_attention_values_with_a_mean_over_long_runs(G):
    """Thousands of entries per warp whose values do not cancel: the sums' roundings must not add up."""
    B, n, n_kv, hd = 32, 131072, 1, 32
    k, v = rows((1, n, n_kv, hd), 386, BF16), rows((1, n, n_kv, hd), 387, BF16, 0.1) + 1
    q = rows((B, 1, n_kv * G, hd), 388)
    c, ref = make(B, G, n_kv, hd, n), Ref(1, G, n_kv, hd, n)
    c.append(0, k.expand(B, n, n_kv, hd), v.expand(B, n, n_kv, hd))
    ref.append(k, v)
    out = torch.empty_like(q)
    c.attention(0, q, out)
    x = torch.einsum("bgd,nd->bgn", q[:, 0].double(), ref.k[0, 0]) / hd ** 0.5
    want = torch.einsum("bgn,nd->bgd", torch.softmax(x, -1), ref.v[0, 0])
    # of a mean near 1: the fp32 rounding of 2^-24 of each partial sum and of the result, a few of each
    assert float((out[:, 0].double() - want).norm() / want.norm()) <= 4 * 2.0 ** -24


def test_non_finite_rows_stay_where_they_are():
    """A NaN in one slot's key, query row or value block poisons only what attends to it."""
    B, n, hd = 4, 70, 64
    k, v = rows((B, n, 1, hd), 25), rows((B, n, 1, hd), 26)
    q = rows((B, 2, 2, hd), 27)
    k[0, 69, 0, 3] = float("nan")             # the last entry: the first query does not see it
    q[1, 1, 1, 7] = float("inf")
    v[2, 69, 0, 40] = float("inf")            # block 1 (dims 32..63) of the last entry
    c, ref = make(B, 2, 1, hd, 96), Ref(B, 2, 1, hd, 96)
    c.append(0, k, v)
    out = torch.empty_like(q)
    c.attention(0, q, out)
    nan = torch.isnan(out)
    assert not nan[0, 0].any() and nan[0, 1].all()
    assert not nan[1, 0].any() and not nan[1, 1, 0].any() and nan[1, 1, 1].all()
    assert not nan[2, 0].any() and not nan[2, 1, :, :32].any() and nan[2, 1, :, 32:].all()
    assert not nan[3].any()
    k[0, 69] = 0
    v[2, 69] = 0
    q[1] = 0
    c.reset()
    ref = Ref(B, 2, 1, hd, 96)
    c.append(0, k, v)
    ref.append(k, v)
    check_attention(c, ref, q)


@pytest.mark.parametrize("n_kv,G,hd,T", [(2, 1, 128, 4), (1, 2, 64, 30), (2, 8, 32, 3), (1, 1, 128, 64)])
@pytest.mark.parametrize("n", [7, 70, 1100])
@pytest.mark.parametrize("small", [False, True])
def test_nan_values_of_the_last_tokens(n_kv, G, hd, T, n, small):
    """NaN blocks among the call's own tokens reach the query tokens behind them, in their 32 dims alone;
    ``small``: beside values of zero and of very unlike sizes."""
    B, cap = 3, 1120
    g = torch.Generator()
    g.manual_seed(396)
    k, v = rows((B, n, n_kv, hd), 397), rows((B, n, n_kv, hd), 398)
    if small:
        v[:, ::3] *= 1e-4
        v[:, 1::5] = 0
    bad = torch.zeros((B, n, n_kv, hd // 32), dtype=torch.bool)
    for b in range(1, B):
        for _ in range(b):
            at = max(0, n - T + int(torch.randint(0, T, (1,), generator=g)))
            bad[b, at, int(torch.randint(0, n_kv, (1,), generator=g)), int(torch.randint(0, hd // 32, (1,), generator=g))] = True
    bad = bad.cuda().repeat_interleave(32, -1)
    c, ref = make(B, n_kv * G, n_kv, hd, cap), Ref(B, n_kv * G, n_kv, hd, cap)
    c.append(0, k, v.masked_fill(bad, float("inf")))
    ref.append(k, v.masked_fill(bad, 0.0))
    for dtype in (F32, BF16):
        q = rows((B, T, n_kv * G, hd), 399, dtype)
        out = torch.empty_like(q)
        c.attention(0, q, out)
        want, tol, _ = ref.attention(q)
        if dtype == BF16:
            tol = tol + want.abs() * 2.0 ** -8 + tol_fp16(ref)
        seen = torch.cumsum(torch.cat([bad.new_zeros((B, T, n_kv, hd)), bad], 1).int(), 1)[:, -T:] > 0   # by query t
        assert torch.equal(torch.isnan(out), seen.repeat_interleave(G, 2))
        assert bool(((out.double() - want).abs() <= tol).logical_or(torch.isnan(out)).all())


@pytest.mark.parametrize("n", [30, 200, 1500, 9000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_nan_value_under_a_weight_of_zero(n, dtype):
    """The first half's weights underflow to 0; 0 times its NaN block is NaN however the work is split."""
    hd = 128
    k, v, q = torch.ones(1, n, 1, hd, device="cuda"), rows((1, n, 1, hd), 31), torch.ones(1, 1, 4, hd, device="cuda")
    k[:, :n // 2] = -1
    v[0, n // 4, 0, 70] = float("nan")        # block 2 (dims 64..95)
    c = make(1, 4, 1, hd, 9024)
    c.append(0, k, v)
    q = (10 * q).to(dtype)
    out = torch.empty_like(q)
    c.attention(0, q, out)
    nan = torch.isnan(out)
    assert nan[..., 64:96].all() and not nan[..., :64].any() and not nan[..., 96:].any()


@pytest.mark.parametrize("n_kv,G,hd,T", [(2, 4, 128, 1), (2, 8, 64, 1), (4, 1, 32, 1), (1, 4, 128, 4)])
def test_attention_is_as_exact_as_plain_fp32(n_kv, G, hd, T):
    """fp32 outputs and weights are no further from the 64-bit result than a plain fp32 computation on
    the same held values is (both errors are random sums: twice the norm, plus one rounding)."""
    B, n = 4, 1500
    c, ref = make(B, n_kv * G, n_kv, hd, 1504, track=T), Ref(B, n_kv * G, n_kv, hd, 1504)
    k, v = rows((B, n, n_kv, hd), 330, BF16), rows((B, n, n_kv, hd), 331, BF16)
    c.append(0, k, v)
    ref.append(k, v)
    q = rows((B, T, n_kv * G, hd), 332, F32, 1.5)
    out = check_attention(c, ref, q, decay=0.0)
    want = ref.attention(q)[0]
    kk, vv = ref.k[:, :, :n].float(), ref.v[:, :, :n].float()
    qq = q.view(B, T, n_kv, G, hd).permute(0, 2, 1, 3, 4)
    x = torch.einsum("bhtgd,bhnd->bhtgn", qq, kk) * hd ** -0.5
    seen = torch.arange(n, device="cuda") < torch.arange(n - T + 1, n + 1, device="cuda")[:, None, None]
    p = torch.softmax(torch.where(seen, x, -torch.inf), -1)
    plain = torch.einsum("bhtgn,bhnd->bhtgd", p, vv).permute(0, 2, 1, 3, 4).reshape(out.shape)
    norm = lambda a: float(a.double().norm())
    assert norm(out - want) <= 2 * norm(plain - want) + 2.0 ** -23 * norm(want)
    w = ref.w[:, :, :n]
    assert norm(c.weights(0)[:, :, :n] - w) <= 2 * norm(p.sum((2, 3)) - w) + 2.0 ** -23 * norm(w)


@pytest.mark.parametrize("n_kv,G,hd,T", [(2, 4, 128, 1), (2, 8, 64, 1), (4, 1, 32, 1), (1, 4, 128, 3), (2, 1, 64, 16)])
@pytest.mark.parametrize("n", [40, 1500, 20000])
def test_bf16_outputs_are_rounded_once(n_kv, G, hd, T, n):
    """A bf16 output is the rounding of a number as near the 64-bit one as an fp32 output's tolerance says,
    and tracked weights have that of fp32 queries."""
    B = 3
    cap = -(-n // 32) * 32
    c, ref = make(B, n_kv * G, n_kv, hd, cap, track=T), Ref(B, n_kv * G, n_kv, hd, cap)
    k, v = rows((B, n, n_kv, hd), 390, BF16), rows((B, n, n_kv, hd), 391, BF16)
    c.append(0, k, v, n_new=i32([n, n // 2, n - 1]))
    ref.append(k, v, [n, n // 2, n - 1])
    q = rows((B, T, n_kv * G, hd), 392, BF16)
    out = check_attention(c, ref, q, decay=0.0)
    want, tol, _ = ref.attention(q)
    assert bool(((out >= (want - tol).to(BF16)) & (out <= (want + tol).to(BF16))).all())
    # an fp32 output of the same queries rounds to the same numbers, but for those next to a border
    full = torch.empty(q.shape, device="cuda")
    c.attention(0, q, full)
    assert float((full.to(BF16) != out).double().mean()) < 1e-2


def test_attention_strided_rows_and_output_over_queries():
    B, T, H, Hkv, hd = 3, 2, 4, 2, 128
    c, ref = make(B, H, Hkv, hd, 128), Ref(B, H, Hkv, hd, 128)
    k, v = rows((B, 120, Hkv, hd), 28), rows((B, 120, Hkv, hd), 29)
    c.append(0, k, v, n_new=i32([120, 77, 1]))
    ref.append(k, v, [120, 77, 1])
    fused = rows((B, T, (H + 2 * Hkv) * hd), 30)
    before = fused.clone()
    q = fused[..., :H * hd].view(B, T, H, hd)
    want, tol, _ = ref.attention(q)
    c.attention(0, q, q)                      # in place
    assert bool(((q.double() - want).abs() <= tol).all())
    assert torch.equal(fused[..., H * hd:], before[..., H * hd:])


# ------------------------------------------------------- weights, eviction
@pytest.mark.parametrize("n_kv,G,hd,T", [(2, 4, 128, 1), (1, 1, 64, 1), (2, 3, 32, 1), (1, 4, 128, 16),
                                         (2, 1, 64, 11)])
def test_weights(n_kv, G, hd, T):
    lens = [0, 1, 31, 100, 515, 1030]
    B, cap = len(lens), 1056
    c, ref = make(B, n_kv * G, n_kv, hd, cap, track=T), Ref(B, n_kv * G, n_kv, hd, cap)
    k, v = rows((B, max(lens), n_kv, hd), 31), rows((B, max(lens), n_kv, hd), 32)
    c.append(0, k, v, n_new=i32(lens))
    ref.append(k, v, lens)
    assert not any(c.weights(0)[b, :, :m].any() for b, m in enumerate(lens))
    before = c.weights(0).clone()
    for i, decay in enumerate((1.0, 1.0, 0.5, 0.0, 1.0)):
        check_attention(c, ref, rows((B, T, n_kv * G, hd), 33 + i, F32, 1.5), decay=decay)
    for b, m in enumerate(lens):              # nothing behind a sequence's end is written
        assert torch.equal(before[b, :, m:].view(torch.int32), c.weights(0)[b, :, m:].view(torch.int32))


def test_decay_zero_does_not_read_old_weights():
    c = make(1, 1, 1, 32, 32, track=1)
    k = rows((1, 20, 1, 32), 40)
    c.append(0, k, k)
    c.weights(0).fill_(float("nan"))
    q, out = rows((1, 1, 1, 32), 41), torch.empty(1, 1, 1, 32, device="cuda")
    c.attention(0, q, out, decay=0.0)
    w = c.weights(0)[0, 0, :20]
    assert abs(float(w.sum()) - 1) < 1e-5
    assert torch.isnan(c.weights(0)[0, 0, 20:]).all()


def fill(c, ref, lens, seed, tie=False):
    B, n = len(lens), max(lens)
    k, v = rows((B, n, ref.Hkv, ref.hd), seed), rows((B, n, ref.Hkv, ref.hd), seed + 1)
    c.append(0, k, v, n_new=i32(lens))
    ref.append(k, v, lens)
    w = rows(tuple(ref.w.shape), seed + 2).abs()
    if tie:
        w = (w * 3).floor()
    c.weights(0).copy_(w)
    ref.w.copy_(w.double())


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (33, 4, 10), (64, 0, 64), (100, 3, 0), (299, 4, 8)])
@pytest.mark.parametrize("tie", [False, True])
def test_evict(hd, budget, sink, recent, tie):
    lens = [0, 1, budget, budget + 1, 300, 150, 299]
    B = len(lens)
    for in_place in (True, False):
        c, ref = make(B, 2, 2, hd, 320), Ref(B, 2, 2, hd, 320)
        fill(c, ref, [min(n, 300) for n in lens], 50, tie)
        d = c if in_place else make(B, 6, 2, hd, 320 if budget > 288 else -(-budget // 32) * 32)
        whole = c.buf.clone()
        c.evict(0, budget, sink, recent, dst=d)
        assert in_place or torch.equal(whole, c.buf)
        ref.evict(budget, sink, recent)
        check_content(d, ref)
        for b, n in enumerate(ref.len):
            assert torch.equal(d.weights(0)[b, :, :n].double(), ref.w[b, :, :n])


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("budget", [1, 33, 79, 95, 96])
def test_evict_in_place_around_the_border(hd, budget):
    """Entries that move within the chunk that holds the budget's border, into it and out of it: in
    place the same as into another cache, and the same each time."""
    B, n_kv = 40, 3
    lens = [min(300, budget + (1, 5, 17, 40, 200)[b % 5]) for b in range(B)]
    c, ref = make(B, n_kv, n_kv, hd, 320), Ref(B, n_kv, n_kv, hd, 320)
    fill(c, ref, lens, 400)
    for b, n in enumerate(lens):              # what lies behind the budget mostly stays
        c.weights(0)[b, :, budget:n] += 2.0 * (b % 3)
        ref.w[b, :, :n].copy_(c.weights(0)[b, :, :n])
    start, d = c.buf.clone(), make(B, n_kv, n_kv, hd, 96)
    c.evict(0, budget, dst=d)
    ref.evict(budget)
    check_content(d, ref)
    for _ in range(3):
        c.buf.copy_(start)
        c.evict(0, budget)
        check_content(c, ref)
        assert torch.equal(c.weights(0)[..., :budget], d.weights(0)[..., :budget])


def test_evict_between_layers_and_equal_weights():
    """Into another layer of the same cache; all weights zero: the first entries stay."""
    c, ref = make(2, 2, 2, 64, 128, n_layer=2), Ref(2, 2, 2, 64, 128)
    k, v = rows((2, 100, 2, 64), 320), rows((2, 100, 2, 64), 321)
    c.append(0, k, v, n_new=i32([100, 70]))
    ref.append(k, v, [100, 70])
    c.evict(0, 64, n_sink=2, n_recent=8, dst_layer=1)
    check_content(c, ref, layer=0)
    ref.evict(64, 2, 8)
    check_content(c, ref, layer=1)
    want = list(range(56)) + list(range(92, 100))
    assert sorted(c.ids(1)[0, 1, :64].tolist()) == want
    # appending goes on behind, with the ids that follow
    c.append(1, k[:, :3], v[:, :3])
    ref.append(k[:, :3], v[:, :3])
    check_content(c, ref, layer=1)
    assert c.ids(1)[0, 0, 64:67].tolist() == [100, 101, 102]


@pytest.mark.parametrize("cap,n,budget", [(1024, 1000, 999), (1056, 1056, 500), (2048, 2048, 31), (4096, 4096, 1000), (8192, 5000, 4999), (20000, 19999, 7000),
                                          (40000, 39001, 20000), (140000, 139999, 33)])
def test_evict_long(cap, n, budget):
    """Capacities of one CTA, of clusters, and of the larger forms; weights exactly alike in places."""
    cap = -(-cap // 32) * 32
    c, ref = make(1, 1, 1, 32, cap), Ref(1, 1, 1, 32, cap)
    fill(c, ref, [n], 60, tie=True)
    c.evict(0, budget, 4, 16)
    ref.evict(budget, 4, 16)
    check_content(c, ref)


def test_evict_odd_weights():
    """Infinite, negative, signed-zero and NaN weights have a fixed order."""
    c, ref = make(1, 1, 1, 32, 32), Ref(1, 1, 1, 32, 32)
    fill(c, ref, [8], 70)
    w = torch.tensor([0.0, -0.0, float("nan"), float("inf"), -1.0, 2.0, -float("inf"), 1.0], device="cuda")
    c.weights(0)[0, 0, :8] = w
    c.evict(0, 4)
    assert c.ids(0)[0, 0, :4].tolist() == [5, 7, 2, 3]   # dropped 0 and 1: 5 and 7 move up
    c.evict(0, 2)
    assert c.ids(0)[0, 0, :2].tolist() == [2, 3]


@pytest.mark.parametrize("cap,n", [(64, 50), (1504, 1500), (9024, 9000)])
def test_evict_takes_zeros_of_both_signs_as_equal(cap, n):
    """0 and -0 are equal weights: the lower index stays, whatever its sign."""
    c, ref = make(2, 2, 2, 32, cap), Ref(2, 2, 2, 32, cap)
    fill(c, ref, [n, n - 3], 410)
    g = torch.Generator(device="cuda")
    g.manual_seed(413)
    u = torch.rand(c.weights(0).shape, generator=g, device="cuda")
    w = torch.where(u < 0.4, 0.0, torch.where(u < 0.9, -0.0, u))
    w[1] = torch.where(u[1] < 0.1, -u[1], w[1])
    c.weights(0).copy_(w)
    ref.w.copy_(w.double())
    c.evict(0, n // 2, 2, 5)
    ref.evict(n // 2, 2, 5)
    check_content(c, ref)


def test_decode_loop_as_used():
    """Prompt, then steps of append, attention with accumulated weights and eviction, in place, on two
    layers; checked against the reference at every step, then replayed from a CUDA graph."""
    B, H, Hkv, hd, cap, budget = 3, 8, 2, 64, 96, 64
    steps = 12
    lens = [60, 5, 80]
    kp, vp = rows((2, B, 80, Hkv, hd), 80), rows((2, B, 80, Hkv, hd), 81)
    ks, vs = rows((steps, 2, B, 1, Hkv, hd), 82, BF16), rows((steps, 2, B, 1, Hkv, hd), 83, BF16)
    qs = rows((steps, 2, B, 1, H, hd), 84, BF16, 2.0)

    def begin(c):
        c.reset()
        for layer in (0, 1):
            c.append(layer, kp[layer], vp[layer], n_new=i32(lens))

    c = make(B, H, Hkv, hd, cap, n_layer=2, track=1)
    refs = [Ref(B, H, Hkv, hd, cap) for _ in (0, 1)]
    begin(c)
    for layer in (0, 1):
        refs[layer].append(kp[layer], vp[layer], lens)
    outs = []
    for i in range(steps):
        for layer, ref in enumerate(refs):
            c.append(layer, ks[i, layer], vs[i, layer])
            ref.append(ks[i, layer], vs[i, layer])
            outs.append(check_attention(c, ref, qs[i, layer], F32, decay=1.0, layer=layer))
            ref.w.copy_(c.weights(layer).double().nan_to_num())   # choose by the kernel's own sums
            c.evict(layer, budget, n_sink=4, n_recent=16)
            ref.evict(budget, 4, 16)
            check_content(c, ref, layer)
    assert c.device_error() == 0

    # the same loop from one captured step; a second cache keeps it apart from the first
    g = make(B, H, Hkv, hd, cap, n_layer=2, track=1)
    begin(g)
    k, v, q = ks[0].clone(), vs[0].clone(), qs[0].clone()
    out = torch.empty((2, B, 1, H, hd), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for layer in (0, 1):
            g.append(layer, k[layer], v[layer])
            g.attention(layer, q[layer], out[layer], decay=1.0)
            g.evict(layer, budget, n_sink=4, n_recent=16)
    for i in range(steps):
        k.copy_(ks[i]); v.copy_(vs[i]); q.copy_(qs[i])
        graph.replay()
        for layer in (0, 1):
            assert torch.equal(out[layer], outs[2 * i + layer])
    for layer in (0, 1):
        check_content(g, refs[layer], layer)
    assert g.device_error() == 0


def test_two_caches_on_two_streams():
    B, H, Hkv, hd, n = 4, 8, 2, 128, 700
    caches, refs, qs, outs = [], [], [], []
    for i in range(2):
        c, ref = make(B, H, Hkv, hd, 704, track=1), Ref(B, H, Hkv, hd, 704)
        k, v = rows((B, n, Hkv, hd), 90 + i), rows((B, n, Hkv, hd), 92 + i)
        c.append(0, k, v)
        ref.append(k, v)
        caches.append(c); refs.append(ref)
        qs.append(rows((B, 1, H, hd), 94 + i)); outs.append(torch.empty(B, 1, H, hd, device="cuda"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for c, q, o, s in zip(caches, qs, outs, streams):
            c.attention(0, q, o, decay=0.0, stream=s)
    torch.cuda.synchronize()
    for ref, q, o in zip(refs, qs, outs):
        want, tol, _ = ref.attention(q)
        assert bool(((o.double() - want).abs() <= tol).all())


def test_a_cache_made_and_used_on_a_side_stream():
    """Creation leaves the workspace ready for any stream: the default one is busy meanwhile, and a
    torch side stream does not wait for it."""
    B, H, Hkv, hd, n = 3, 8, 2, 64, 1500
    ref = Ref(B, H, Hkv, hd, 1504)
    k, v, q = rows((B, n, Hkv, hd), 350), rows((B, n, Hkv, hd), 351), rows((B, 1, H, hd), 352)
    ref.append(k, v)
    want, tol, wtol = ref.attention(q, 0.0)
    a = torch.randn(4096, 4096, device="cuda")
    s = torch.cuda.Stream()
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    for _ in range(100):
        a = (a @ a).clamp(-1, 1)
    with torch.cuda.stream(s):
        c = pnb.Kv4Cache(1, B, H, Hkv, hd, 1504, track=1)
        c.reset()
        c.append(0, k, v)
        c.attention(0, q, out, decay=0.0)
        c.evict(0, 1000, 4, 100)
    torch.cuda.synchronize()
    assert bool(((out.double() - want).abs() <= tol).all())
    assert c.lengths(0).tolist() == [1000] * B and c.device_error() == 0
    assert float(c.weights(0)[:, :, :1000].sum()) <= B * H * (1 + wtol)


def test_a_copied_buffer_is_a_copied_cache():
    c, ref = make(2, 4, 2, 64, 64), Ref(2, 4, 2, 64, 64)
    k, v = rows((2, 50, 2, 64), 96), rows((2, 50, 2, 64), 97)
    c.append(0, k, v, n_new=i32([50, 9]))
    ref.append(k, v, [50, 9])
    d = pnb.Kv4Cache(1, 2, 4, 2, 64, 64, buf=c.buf.clone())
    c.reset()
    check_content(d, ref)
    check_attention(d, ref, rows((2, 1, 4, 64), 98))


def test_wild_lengths_in_the_buffer_stay_inside_it():
    c = make(2, 2, 1, 32, 32, track=1)
    k = rows((2, 32, 1, 32), 99)
    c.append(0, k, k)
    c.lengths(0).copy_(i32([1 << 30, -5]))
    q, out = rows((2, 1, 2, 32), 100), torch.empty(2, 1, 2, 32, device="cuda")
    c.attention(0, q, out, decay=0.0)
    assert torch.isfinite(out).all() and not out[1].any() and out[0].any()


def test_after_a_models_prefill():
    """A prefilled state's K / V of one layer moved into a 4-bit cache, and the step's own rotated
    queries answered from it: the held values are the state's cache through the quantiser."""
    import synth.workloads as wl
    from synth import BF16 as SBF16

    s = wl.Shape(n_vocab=1000, n_embd=1024, n_head=8, n_kv_head=2, n_layer=2, n_ff=1024, n_ctx=96,
                 rope_theta=1e4, rms_norm_eps=1e-5, sliding_window=0, dtype=SBF16)
    sm = pnb.SynthModel(s, 21, device="cuda")
    st = sm.new_state()
    prompt = torch.arange(1, 71, dtype=torch.int32, device="cuda")
    st.prefill(prompt)
    torch.cuda.synchronize()
    kv = st.kv.view(torch.uint8)[:sm.model.kv_bytes()].view(BF16).view(2, 2, 1, 2, 96, 128)
    c, ref = make(1, 8, 2, 128, 96, n_layer=2), Ref(1, 8, 2, 128, 96)
    k, v = kv[1, 0].transpose(1, 2)[:, :70], kv[1, 1].transpose(1, 2)[:, :70]
    c.append(1, k, v)
    ref.append(k, v)
    check_content(c, ref, layer=1)

    class Holder:
        __cuda_array_interface__ = {"shape": (1, 1, 8, 128), "typestr": "<f4",
                                    "data": (st.activations()["q"], False), "version": 3}
    st.run_kernel(pnb.PNB_KERNEL_QKV, 1)
    q = torch.as_tensor(Holder(), device="cuda").clone()
    check_attention(c, ref, q, layer=1)


# ---------------------------------------------------------------- refusals
def test_refusals():
    c = make(2, 4, 2, 64, 64, n_layer=2, track=1)
    k, q = rows((2, 3, 2, 64), 101), rows((2, 1, 4, 64), 102)
    out = torch.empty_like(q)

    def code(f, *a, **kw):
        with pytest.raises(pnb.PnbError) as e:
            f(*a, **kw)
        return e.value.code

    assert code(c.append, 2, k, k) == -1 and code(c.append, -1, k, k) == -1
    assert code(c.append, 0, k[:, :, :1], k[:, :, :1]) == -1
    assert code(c.append, 0, k, k[:, :2]) == -1
    assert code(c.append, 0, k, k.to(BF16)) == -1
    assert code(c.append, 0, k.half(), k.half()) == -1
    assert code(c.append, 0, k.cpu(), k.cpu()) == -10
    assert code(c.append, 0, k[..., ::2].expand(2, 3, 2, 32), k) == -1
    odd = torch.empty(2, 3, 2 * 64 + 1, device="cuda")[..., :128].view(2, 3, 2, 64)
    assert code(c.append, 0, odd, odd) == -3                      # rows not 16-byte aligned
    assert code(c.append, 0, rows((2, 65, 2, 64), 1), rows((2, 65, 2, 64), 1)) == -1
    assert code(c.append, 0, k, k, n_new=torch.zeros(2, device="cuda")) == -1
    assert code(c.append, 0, k, k, start=i32([0])) == -1
    assert code(c.read, 0, k[:1].expand(2, 3, 2, 64), k.clone()) == -1   # overlapping outputs
    assert code(c.attention, 0, q, out, decay=-0.5) == -1
    assert code(c.attention, 0, q, out, decay=float("nan")) == -1
    assert code(c.attention, 0, q, out, decay=float("inf")) == -1
    q2 = rows((2, 2, 4, 64), 103)
    assert code(c.attention, 0, q2, q2.clone(), decay=1.0) == -1          # more tokens than `track`
    q33 = rows((2, 33, 4, 64), 103)
    assert code(c.attention, 0, q33, q33.clone()) == -5                   # 66 rows per KV head
    assert code(c.attention, 0, q[:, :0], out[:, :0]) == -1
    assert code(c.attention, 0, q, out[:1].expand(2, 1, 4, 64)) == -1
    assert code(c.evict, 0, 0) == -1 and code(c.evict, 0, 65) == -1
    assert code(c.evict, 0, 10, n_sink=6, n_recent=5) == -1
    assert code(c.evict, 0, 10, n_sink=-1) == -1
    assert code(c.evict, 0, 10, dst_layer=2) == -1
    assert code(c.evict, 0, 10, dst=make(2, 4, 2, 32, 64)) == -1
    assert code(c.evict, 0, 33, dst=make(2, 4, 2, 64, 32)) == -1
    assert code(c.evict, 0, 10, dst=pnb.Kv4Cache(1, 2, 4, 2, 64, 32, buf=c.buf)) == -1
    assert code(c.reset, 2) == -1
    cfg = dict(n_layer=1, n_slot=1, n_head=1, n_kv_head=1, head_dim=32, cap=32)
    assert code(pnb.Kv4Cache, **cfg, buf=torch.zeros(1 << 16, dtype=torch.uint8)) == -10   # host memory
    dev = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    assert code(pnb.Kv4Cache, **cfg, buf=dev.view(-1, 2)[:, 0]) == -1
    assert code(pnb.Kv4Cache, **cfg, buf=dev[:1024]) == -1                # too small
    assert code(pnb.Kv4Cache, **cfg, buf=dev[64:]) == -3                  # not 128-byte aligned
    assert code(pnb.Kv4Cache, **{**cfg, "head_dim": 48}) == -5
    big = pnb.Kv4Cache(1, 1, 1, 1, 32, (1 << 18) + 32)
    big.reset()
    assert code(big.evict, 0, 10) == -5
    assert c.device_error() == 0 and c.lengths(0).tolist() == [0, 0]


def test_numbers_past_32_bits_are_refused():
    """They would reach the library modulo 2^32: another layer, a budget of 5, a small cache."""
    c, k, q = make(2, 2, 1, 32, 64, n_layer=2, track=1), rows((2, 40, 1, 32), 420), rows((2, 1, 2, 32), 421)
    c.append(0, k, k)
    before, wrap = c.buf.clone(), 1 << 32

    def refused(f, *a, **kw):
        with pytest.raises(pnb.PnbError) as e:
            f(*a, **kw)
        return e.value.code == -1

    assert refused(c.append, wrap, k, k) and refused(c.read, wrap, k.clone(), k.clone())
    assert refused(c.attention, wrap, q, q.clone(), decay=1.0) and refused(c.lengths, wrap)
    assert refused(c.evict, wrap, 5) and refused(c.evict, 0, wrap + 5) and refused(c.evict, 0, 5, dst_layer=wrap + 1)
    assert refused(c.evict, 0, 5, n_sink=wrap) and refused(c.evict, 0, 5, n_recent=wrap)
    assert refused(c.reset, wrap) and refused(c.reset, -1) and refused(c.reset, 2)
    assert torch.equal(before, c.buf)
    cfg = dict(n_layer=1, n_slot=1, n_head=1, n_kv_head=1, head_dim=32, cap=32)
    for name in cfg:
        assert refused(pnb.Kv4Cache, **{**cfg, name: cfg[name] + wrap})


def test_rows_over_one_another_are_refused():
    """read's K over its V, attention's output over others' queries, eviction between overlapping buffers."""
    B, T, H, Hkv, hd = 2, 3, 4, 2, 64
    c = make(B, H, Hkv, hd, 64)
    c.append(0, rows((B, 40, Hkv, hd), 104), rows((B, 40, Hkv, hd), 105))
    want = torch.empty(2, B, T, Hkv, hd, device="cuda")
    c.read(0, want[0], want[1])

    def refused(f, *a, **kw):
        with pytest.raises(pnb.PnbError) as e:
            f(*a, **kw)
        return e.value.code == -1

    flat = torch.zeros(1 << 14, device="cuda")
    at = lambda off, s, dtype=F32: flat.view(dtype)[off:].as_strided((B, T, Hkv, hd), s)
    plain = (T * Hkv * hd, Hkv * hd, hd, 1)
    n = B * T * Hkv * hd
    for off in (0, 16, hd, hd * Hkv, n - hd, n - 4):          # rows over rows, whole or in part
        assert refused(c.read, 0, at(0, plain), at(off, plain))
        assert refused(c.read, 0, at(off, plain), at(0, plain))
    side = (2 * T * Hkv * hd, 2 * Hkv * hd, hd, 1)             # K and V of a token side by side
    pair = (2 * T * Hkv * hd, 2 * Hkv * hd, 2 * hd, 1)         # of a head
    by_head = (Hkv * 2 * T * hd, hd, 2 * T * hd, 1)            # tokens inside heads
    for s, off in ((plain, n), (side, Hkv * hd), (pair, hd), (by_head, T * hd)):
        for a, b in ((0, off), (off, 0)):
            k, v = at(a, s), at(b, s)
            flat.zero_()
            c.read(0, k, v)
            assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    for s, off in ((side, hd), (pair, hd // 2), (pair, 2 * hd), (by_head, hd), (by_head, 2 * T * hd)):
        assert refused(c.read, 0, at(0, s), at(off, s)) and refused(c.read, 0, at(off, s), at(0, s))
    assert refused(c.read, 0, at(0, pair), at(hd, side))       # between one another, strides differ

    q = flat[:B * T * H * hd].view(B, T, H, hd)
    shifted = flat[hd:hd + B * T * H * hd].view(B, T, H, hd)
    assert refused(c.attention, 0, q, shifted) and refused(c.attention, 0, shifted, q)
    assert refused(c.attention, 0, q, flat.view(BF16)[:q.numel()].view(B, T, H, hd))
    assert refused(c.attention, 0, q, flat.as_strided((B, T, H, hd), (H * hd, B * H * hd, hd, 1)))
    c.attention(0, q, q)

    nbytes = c.buf.numel()
    two = torch.empty(2 * nbytes, dtype=torch.uint8, device="cuda")
    over = [pnb.Kv4Cache(1, B, H, Hkv, hd, 64, buf=two[o:o + nbytes]) for o in (0, 128, nbytes)]
    over[0].reset()
    assert refused(over[0].evict, 0, 8, dst=over[1]) and refused(over[1].evict, 0, 8, dst=over[0])
    over[0].evict(0, 8, dst=over[2])
    assert over[2].lengths(0).tolist() == [0, 0]
