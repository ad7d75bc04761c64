"""The paged KV cache's C ABI: sizes and host-side refusals (no GPU needed)."""
import ctypes

import pytest

import transformer_decode_step_gb300 as pnb


def _cfg(**kw):
    base = dict(n_layer=2, n_page=5, page=64, n_head=8, n_kv_head=4, head_dim=64, shared_tok=0, rope_neox=0,
                rope_section=(0, 0, 0), rope_theta=10000.0)
    base.update(kw)
    base["rope_section"] = (ctypes.c_int32 * 3)(*base["rope_section"])
    return pnb.pnb_pkv_config(**base)


def _new(c, buf=1 << 20, bytes_=1 << 60):
    h = ctypes.c_void_p()
    rc = pnb.pnb_pkv_new(ctypes.byref(c), buf, bytes_, ctypes.byref(h))
    assert h.value is None
    return rc


def test_pool_bytes():
    assert pnb.pnb_pkv_bytes(ctypes.byref(_cfg())) == 2 * 5 * 2 * 4 * 64 * 64 * 2
    assert pnb.pnb_pkv_bytes(ctypes.byref(_cfg(page=16, head_dim=128, n_layer=1))) == 5 * 2 * 4 * 16 * 128 * 2
    # past 32 bits
    big = _cfg(n_layer=80, n_page=100000, page=128, head_dim=128, n_kv_head=8, n_head=8)
    assert pnb.pnb_pkv_bytes(ctypes.byref(big)) == 80 * 100000 * 2 * 8 * 128 * 128 * 2


@pytest.mark.parametrize("bad", [
    dict(n_layer=0), dict(n_page=0), dict(n_head=0), dict(n_kv_head=0), dict(n_kv_head=3), dict(shared_tok=-1),
    dict(rope_neox=2), dict(rope_section=(8, 8, 8)), dict(rope_section=(40, -8, 0)), dict(rope_theta=-1.0),
    dict(rope_theta=float("nan")), dict(rope_theta=float("inf")),
])
def test_invalid_configs(bad):
    assert pnb.pnb_pkv_bytes(ctypes.byref(_cfg(**bad))) == 0
    assert _new(_cfg(**bad)) == -1


@pytest.mark.parametrize("bad", [
    dict(head_dim=32), dict(head_dim=96), dict(head_dim=256), dict(page=8), dict(page=48), dict(page=256), dict(page=0),
    dict(n_head=260), dict(n_page=1 << 30), dict(n_layer=5000), dict(shared_tok=1 << 28),
])
def test_unsupported_configs(bad):
    assert pnb.pnb_pkv_bytes(ctypes.byref(_cfg(**bad))) == 0
    assert _new(_cfg(**bad)) == -5


def test_new_checks_its_buffer():
    c = _cfg()
    n = pnb.pnb_pkv_bytes(ctypes.byref(c))
    h = ctypes.c_void_p()
    assert pnb.pnb_pkv_new(None, 1 << 20, n, ctypes.byref(h)) == -2
    assert pnb.pnb_pkv_new(ctypes.byref(c), None, n, ctypes.byref(h)) == -2
    assert pnb.pnb_pkv_new(ctypes.byref(c), 1 << 20, n, None) == -2
    assert _new(c, (1 << 20) + 64, n) == -3
    assert _new(c, 1 << 20, n - 1) == -1


def test_null_handles():
    rows = pnb.pnb_rows(1 << 20, 0, 0, 0, 0)
    b = pnb.pnb_pkv_batch(1, 1, None, 1 << 20, 1 << 20)
    r = ctypes.byref
    assert pnb.pnb_pkv_bytes(None) == 0
    assert pnb.pnb_pkv_append(None, 0, r(b), 1, r(rows), r(rows), None, None, None, None) == -2
    assert pnb.pnb_pkv_attention(None, 0, r(b), 1, r(rows), r(rows), 0, None) == -2
    assert pnb.pnb_pkv_attention_shared(None, 0, r(b), 1, None, None, 1, r(rows), r(rows), 0, None) == -2
    assert pnb.pnb_pkv_check(None, None) == -2
    pnb.pnb_pkv_free(None)
