"""Calls of the paged KV cache at the ends of what its header allows, against 64 bits.

Cases, oracle and tolerances are those of the cache's other tests (test_gpu_paged.py).
"""
import math

import pytest
import torch

import transformer_decode_step_gb300 as pnb
from test_gpu_paged import Case, _wide

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
