"""The 4-bit KV cache's C ABI: sizes and host-side refusals (no GPU needed)."""
import ctypes

import pytest

import transformer_decode_step_gb300 as pnb


def _cfg(**kw):
    base = dict(n_layer=2, n_slot=3, n_head=8, n_kv_head=4, head_dim=64, cap=96, track=1)
    base.update(kw)
    return pnb.pnb_kvq_config(**base)


def _bytes(cfg):
    return int(pnb.pnb_kvq_bytes(ctypes.byref(cfg)))


def test_buffer_bytes():
    # per layer: 36 bytes per 64 values (32 bytes of codes, two fp16 scales), K and V; an id
    # and a weight per entry; a length and a count per slot; each part padded to 256 bytes
    up = lambda n: (n + 255) // 256 * 256
    entries = 3 * 4 * 96
    layer = up(entries * 2 * 36) + 2 * up(entries * 4) + 2 * up(3 * 4)
    assert _bytes(_cfg()) == 2 * layer
    # 144 bytes of codes and scales per position and KV head at head_dim 128
    big = _bytes(_cfg(n_layer=1, n_slot=1, n_kv_head=1, n_head=1, head_dim=128, cap=1 << 20))
    assert big == (1 << 20) * (144 + 8) + 512


@pytest.mark.parametrize("bad", [
    dict(n_layer=0), dict(n_slot=0), dict(n_head=0), dict(n_kv_head=0), dict(cap=0),
    dict(cap=97), dict(cap=-32), dict(track=-1), dict(n_kv_head=3),
])
def test_invalid_configs(bad):
    c = _cfg(**bad)
    assert _bytes(c) == 0
    h = ctypes.c_void_p()
    assert pnb.pnb_kvq_new(ctypes.byref(c), 1 << 20, 1 << 40, ctypes.byref(h)) == -1
    assert h.value is None


@pytest.mark.parametrize("bad", [
    dict(head_dim=96), dict(head_dim=256), dict(n_slot=1025), dict(n_head=260, n_kv_head=4),
    dict(track=33), dict(cap=(1 << 20) + 32), dict(n_slot=1024, n_kv_head=64, n_head=64, cap=1 << 20),
])
def test_unsupported_configs(bad):
    c = _cfg(**bad)
    assert _bytes(c) == 0
    h = ctypes.c_void_p()
    assert pnb.pnb_kvq_new(ctypes.byref(c), 1 << 20, 1 << 60, ctypes.byref(h)) == -5


def test_new_checks_its_buffer():
    c = _cfg()
    h = ctypes.c_void_p()
    r = ctypes.byref
    assert pnb.pnb_kvq_new(None, 1 << 20, _bytes(c), r(h)) == -2
    assert pnb.pnb_kvq_new(r(c), None, _bytes(c), r(h)) == -2
    assert pnb.pnb_kvq_new(r(c), 1 << 20, _bytes(c), None) == -2
    assert pnb.pnb_kvq_new(r(c), (1 << 20) + 64, _bytes(c), r(h)) == -3
    assert pnb.pnb_kvq_new(r(c), 1 << 20, _bytes(c) - 1, r(h)) == -1


def test_null_handles():
    rows = pnb.pnb_rows(1 << 20, 0, 0, 0, 0)
    r = ctypes.byref
    assert pnb.pnb_kvq_bytes(None) == 0
    assert pnb.pnb_kvq_reset(None, -1, None) == -2
    assert pnb.pnb_kvq_append(None, 0, r(rows), r(rows), 1, None, None, None) == -2
    assert pnb.pnb_kvq_read(None, 0, None, 1, r(rows), r(rows), None) == -2
    assert pnb.pnb_kvq_attention(None, 0, r(rows), 1, r(rows), -1.0, None) == -2
    assert pnb.pnb_kvq_evict(None, 0, None, 0, 1, 0, 0, None) == -2
    assert pnb.pnb_kvq_layer_views(None, 0, None) == -2
    assert pnb.pnb_kvq_check(None, None) == -2
    pnb.pnb_kvq_free(None)
