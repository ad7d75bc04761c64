"""The 4-bit KV cache (pnb_kvq_*, include/pnb.h): append, read, attention, eviction.

Like the rest of the binding it only marshals arguments.  The cache's buffer is
a torch tensor; lengths, ids and weights are views of it.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

from . import (PNB_BF16, PNB_F32, PnbError, _ptr, check, pnb_kvq_append, pnb_kvq_attention,
               pnb_kvq_bytes, pnb_kvq_check, pnb_kvq_config, pnb_kvq_evict, pnb_kvq_free,
               pnb_kvq_layer_views, pnb_kvq_new, pnb_kvq_read, pnb_kvq_reset, pnb_kvq_views)

# a pnb_rows as bytes (a ctypes.Structure takes three times as long to fill, and a
# short attention call is bound by the host)
_pack_rows = struct.Struct("@Pqqqi4x").pack


def _i32(v, what: str) -> int:
    """v itself, refused where ctypes would cut it down to 32 bits."""
    if not -(1 << 31) <= v < 1 << 31:
        raise PnbError(-1, f"{what} {v} does not fit 32 bits")
    return v


class Kv4Cache:
    """A pnb_kvq over a torch buffer (``buf``, allocated if None; reset() a new one).

    Row tensors (k, v, q, out) are [n_slot][T][heads][head_dim], fp32 or bf16,
    head_dim contiguous, other strides free as long as rows stay 16-byte aligned."""

    def __init__(self, n_layer: int, n_slot: int, n_head: int, n_kv_head: int, head_dim: int,
                 cap: int, track: int = 0, buf=None, device=None):
        import torch

        self._h = None
        self.cfg = pnb_kvq_config(*(_i32(v, f"Kv4Cache: {n}") for v, n in zip(
            (n_layer, n_slot, n_head, n_kv_head, head_dim, cap, track),
            ("n_layer", "n_slot", "n_head", "n_kv_head", "head_dim", "cap", "track"))))
        self._dtypes = {torch.float32: PNB_F32, torch.bfloat16: PNB_BF16}
        self._int32 = torch.int32
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        nbytes = int(pnb_kvq_bytes(ctypes.byref(self.cfg)))
        if buf is None:
            buf = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device or "cuda")
        if not buf.is_cuda or buf.get_device() != torch.cuda.current_device():
            raise PnbError(-10, f"Kv4Cache: the buffer is on {buf.device}, not on the current CUDA device")
        if not buf.is_contiguous():
            raise PnbError(-1, "Kv4Cache: the buffer is not contiguous")
        self.buf = buf
        h = ctypes.c_void_p()
        check(pnb_kvq_new(ctypes.byref(self.cfg), _ptr(buf), buf.numel() * buf.element_size(),
                          ctypes.byref(h)), "pnb_kvq_new")
        self._h = h.value
        self._device = buf.get_device()
        self._n_slot, self._head_dim, self._slots = n_slot, head_dim, (n_slot,)
        self._n_head, self._n_kv = n_head, n_kv_head
        self._views = {}

    def __del__(self):
        if getattr(self, "_h", None):
            pnb_kvq_free(self._h)
            self._h = None

    @property
    def handle(self) -> int:
        return self._h

    def _stream(self, stream) -> int:
        """A stream's handle; by default the current one of the cache's device."""
        if stream is None:
            return self._raw_stream(self._device)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _shape(self, t, what: str, heads: int) -> tuple:
        """[n_slot][T][heads][head_dim] with T from the tensor."""
        shape = t.shape
        if len(shape) != 4:
            raise PnbError(-1, f"{what}: needs rows [n_slot][T][heads][head_dim]")
        return (self._n_slot, shape[1], heads, self._head_dim)

    def _rows(self, t, what: str, shape: tuple) -> bytes:
        if t.shape != shape:
            raise PnbError(-1, f"{what}: shape {tuple(t.shape)} is not {shape}")
        dt = self._dtypes.get(t.dtype)
        slot, token, head, one = t.stride()
        if dt is None or one != 1:
            raise PnbError(-1, f"{what}: needs fp32 or bf16 rows with head_dim contiguous")
        if t.get_device() != self._device:
            raise PnbError(-10, f"{what}: on {t.device}, the cache is on {self.buf.device}")
        # a dimension of one element has no stride of its own
        n, T, heads, _ = shape
        return _pack_rows(t.data_ptr(), slot if n > 1 else 0, token if T > 1 else 0,
                          head if heads > 1 else 0, dt)

    def _ints(self, t, what: str):
        if t is None:
            return None
        if t.dtype != self._int32 or t.shape != self._slots or not t.is_contiguous() \
                or t.get_device() != self._device:
            raise PnbError(-1, f"{what}: needs {self._n_slot} contiguous int32 on the cache's device")
        return t.data_ptr()

    def reset(self, slot: Optional[int] = None, stream=None):
        """Empty one slot, or all of them (which also clears the error bits), in every layer."""
        if slot is not None and not 0 <= slot < self._n_slot:
            raise PnbError(-1, f"reset: slot {slot} of {self._n_slot}")
        check(pnb_kvq_reset(self._h, -1 if slot is None else slot, self._stream(stream)), "pnb_kvq_reset")

    def append(self, layer: int, k, v, n_new=None, start=None, stream=None):
        """Quantise and append n_new[b] (default: all T) rows of every slot b at entry
        start[b] (default: its length).  n_new, start: device int32 [n_slot]."""
        shape = self._shape(k, "k", self._n_kv)
        check(pnb_kvq_append(self._h, _i32(layer, "layer"), self._rows(k, "k", shape), self._rows(v, "v", shape),
                             shape[1], self._ints(n_new, "n_new"), self._ints(start, "start"),
                             self._stream(stream)), "pnb_kvq_append")

    def read(self, layer: int, k, v, first=None, stream=None):
        """Write the values of entries first[b] (default 0) .. + T - 1 into k and v."""
        shape = self._shape(k, "k", self._n_kv)
        check(pnb_kvq_read(self._h, _i32(layer, "layer"), self._ints(first, "first"), shape[1],
                           self._rows(k, "k", shape), self._rows(v, "v", shape),
                           self._stream(stream)), "pnb_kvq_read")

    def attention(self, layer: int, q, out, decay: Optional[float] = None, stream=None):
        """Attention of the last T appended tokens' queries into ``out``; with ``decay``,
        weights = decay * weights + this call's softmax weights."""
        shape = self._shape(q, "q", self._n_head)
        if decay is None:
            decay = -1.0
        elif not decay >= 0.0:
            raise PnbError(-1, f"decay {decay} is negative or not a number")
        check(pnb_kvq_attention(self._h, _i32(layer, "layer"), self._rows(q, "q", shape), shape[1],
                                self._rows(out, "out", shape), decay, self._stream(stream)),
              "pnb_kvq_attention")

    def evict(self, layer: int, budget: int, n_sink: int = 0, n_recent: int = 0,
              dst: Optional["Kv4Cache"] = None, dst_layer: Optional[int] = None, stream=None):
        """Keep at most ``budget`` entries per slot and KV head, in place or into
        (dst, dst_layer); see pnb_kvq_evict for which."""
        d = self if dst is None else dst
        check(pnb_kvq_evict(self._h, _i32(layer, "layer"), d._h,
                            layer if dst_layer is None else _i32(dst_layer, "dst_layer"), _i32(budget, "budget"),
                            _i32(n_sink, "n_sink"), _i32(n_recent, "n_recent"), self._stream(stream)),
              "pnb_kvq_evict")

    def _view(self, layer: int, name: str):
        import torch

        key = (layer, name)
        if key not in self._views:
            v = pnb_kvq_views()
            check(pnb_kvq_layer_views(self._h, _i32(layer, "layer"), ctypes.byref(v)), "pnb_kvq_layer_views")
            g = self.cfg
            shape = (g.n_slot,) if name in ("len", "seen") else (g.n_slot, g.n_kv_head, g.cap)
            n = 1
            for s in shape:
                n *= s
            at = getattr(v, name) - self.buf.data_ptr()
            flat = self.buf.view(-1).view(torch.uint8)[at:at + 4 * n]
            self._views[key] = flat.view(torch.float32 if name == "weights" else torch.int32).view(shape)
        return self._views[key]

    def lengths(self, layer: int):
        """Entries held per slot (int32 [n_slot], a view of the buffer)."""
        return self._view(layer, "len")

    def seen(self, layer: int):
        """Tokens ever appended per slot, the next entry's id (int32 [n_slot])."""
        return self._view(layer, "seen")

    def ids(self, layer: int):
        """Original position of every entry (int32 [n_slot][n_kv_head][cap])."""
        return self._view(layer, "ids")

    def weights(self, layer: int):
        """Accumulated attention weight of every entry (fp32 [n_slot][n_kv_head][cap])."""
        return self._view(layer, "weights")

    def device_error(self) -> int:
        """Synchronise and read the device error bits (PNB_DEV_ERR_*)."""
        e = ctypes.c_int32()
        rc = pnb_kvq_check(self._h, ctypes.byref(e))
        if rc not in (0, -8):
            check(rc, "pnb_kvq_check")
        return e.value
