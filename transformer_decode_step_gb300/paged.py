"""The paged KV cache (pnb_pkv_*, include/pnb.h): append with rotation, attention of packed
sequences, attention of sequences that share a prefix.

Like the rest of the binding it only marshals arguments.  The pool is a torch tensor; page
tables, lengths and token counts are the caller's device tensors, read when a call runs on the
device (so a captured call answers for what they hold at its replay).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

from . import (PNB_BF16, PNB_F32, PnbError, _ptr, check, pnb_pkv_append, pnb_pkv_attention,
               pnb_pkv_attention_shared, pnb_pkv_batch, pnb_pkv_bytes, pnb_pkv_check, pnb_pkv_config, pnb_pkv_free,
               pnb_pkv_new)
from .kv4 import _i32, _pack_rows


class PagedBatch:
    """The sequences of a call: device int32 tensors ``lens`` [n_seq], ``pages`` [n_seq][max_page]
    and ``start`` [n_seq + 1] (None: every sequence has the same number of tokens)."""

    def __init__(self, kv: "PagedKv", lens, pages, start=None):
        if lens.dim() != 1 or lens.numel() < 1:
            raise PnbError(-1, "lens: needs [n_seq] int32")
        n = lens.numel()
        if pages.dim() != 2 or pages.shape[0] != n or pages.shape[1] < 1:
            raise PnbError(-1, f"pages: shape {tuple(pages.shape)} is not ({n}, max_page)")
        if start is not None and start.shape != (n + 1,):
            raise PnbError(-1, f"start: shape {tuple(start.shape)} is not ({n + 1},)")
        self.n_seq = n
        self.tensors = (lens, pages, start)
        kv._ints(lens, "lens")
        kv._ints(pages, "pages")
        self._c = pnb_pkv_batch(n, _i32(pages.shape[1], "max_page"),
                                None if start is None else kv._ints(start, "start"), lens.data_ptr(),
                                pages.data_ptr())
        self._ref = ctypes.addressof(self._c)


class PagedKv:
    """A pnb_pkv over a torch buffer (``buf``, a zeroed one if None).

    Row tensors (q, k, v, out) are [n_tok][heads][head_dim], fp32 or bf16, head_dim contiguous,
    other strides free as long as rows stay 16-byte aligned."""

    def __init__(self, n_layer: int, n_head: int, n_kv_head: int, head_dim: int, n_page: int, page: int = 64,
                 rope_theta: float = 10000.0, rope_neox: bool = False,
                 rope_sections: Optional[Sequence[int]] = None, shared_tok: int = 0, buf=None, device=None):
        import torch

        self._h = None
        sections = tuple(rope_sections) if rope_sections is not None else (0, 0, 0)
        if len(sections) != 3:
            raise PnbError(-1, f"PagedKv: rope_sections {sections} are not three")
        names = ("n_layer", "n_page", "page", "n_head", "n_kv_head", "head_dim", "shared_tok")
        ints = [_i32(v, f"PagedKv: {n}") for v, n in
                zip((n_layer, n_page, page, n_head, n_kv_head, head_dim, shared_tok), names)]
        self.cfg = pnb_pkv_config(*ints, 1 if rope_neox else 0,
                                  (ctypes.c_int32 * 3)(*(_i32(v, "PagedKv: rope_sections") for v in sections)),
                                  rope_theta)
        self._dtypes = {torch.float32: PNB_F32, torch.bfloat16: PNB_BF16}
        self._int32 = torch.int32
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        nbytes = int(pnb_pkv_bytes(ctypes.byref(self.cfg)))
        if buf is None:
            buf = torch.zeros(max(nbytes, 1), dtype=torch.uint8, device=device or "cuda")
        if not buf.is_cuda or buf.get_device() != torch.cuda.current_device():
            raise PnbError(-10, f"PagedKv: the buffer is on {buf.device}, not on the current CUDA device")
        if not buf.is_contiguous():
            raise PnbError(-1, "PagedKv: the buffer is not contiguous")
        self.buf = buf
        h = ctypes.c_void_p()
        check(pnb_pkv_new(ctypes.byref(self.cfg), _ptr(buf), buf.numel() * buf.element_size(), ctypes.byref(h)),
              "pnb_pkv_new")
        self._h = h.value
        self._device = buf.get_device()
        self._n_head, self._n_kv, self._hd = n_head, n_kv_head, head_dim
        shape = (n_layer, n_page, 2, n_kv_head, page, head_dim)
        flat = buf.view(-1).view(torch.uint8)[:nbytes].view(torch.bfloat16)
        self._pages = flat.view(shape)

    def __del__(self):
        if getattr(self, "_h", None):
            pnb_pkv_free(self._h)
            self._h = None

    @property
    def handle(self) -> int:
        return self._h

    def pages(self, layer: int):
        """A layer's pages, bf16 [n_page][2 (K, V)][n_kv_head][page][head_dim], a view of the buffer."""
        return self._pages[layer]

    def batch(self, lens, pages, start=None) -> PagedBatch:
        """The sequences of a call (PagedBatch); good for any number of calls and layers."""
        return PagedBatch(self, lens, pages, start)

    def _stream(self, stream) -> int:
        """A stream's handle; by default the current one of the cache's device."""
        if stream is None:
            return self._raw_stream(self._device)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _ints(self, t, what: str):
        if t.dtype != self._int32 or not t.is_contiguous() or t.get_device() != self._device:
            raise PnbError(-1, f"{what}: needs contiguous int32 on the cache's device")
        return t.data_ptr()

    def _rows(self, t, what: str, n_tok: int, heads: int) -> bytes:
        if t.shape != (n_tok, heads, self._hd):
            raise PnbError(-1, f"{what}: shape {tuple(t.shape)} is not {(n_tok, heads, self._hd)}")
        dt = self._dtypes.get(t.dtype)
        token, head, one = t.stride()
        if dt is None or one != 1:
            raise PnbError(-1, f"{what}: needs fp32 or bf16 rows with head_dim contiguous")
        if t.get_device() != self._device:
            raise PnbError(-10, f"{what}: on {t.device}, the cache is on {self.buf.device}")
        # a dimension of one element has no stride of its own
        return _pack_rows(t.data_ptr(), 0, token if n_tok > 1 else 0, head if heads > 1 else 0, dt)

    def _batch(self, b) -> int:
        if not isinstance(b, PagedBatch):
            raise PnbError(-1, "batch: needs a PagedBatch")
        return b._ref

    def append(self, layer: int, batch: PagedBatch, k, v, q=None, q_out=None, pos=None, stream=None):
        """Rotate and store the tokens' keys, store their values; with ``q`` write the rotated
        queries to ``q_out`` (None: over ``q``).  ``pos``: int32 [n_tok], or [3][n_tok] with
        rope_sections; None: a token's entry index."""
        n = _i32(k.shape[0], "tokens")
        if pos is not None:
            three = self.cfg.rope_section[0] or self.cfg.rope_section[1] or self.cfg.rope_section[2]
            if pos.shape != ((3, n) if three else (n,)):
                raise PnbError(-1, f"pos: shape {tuple(pos.shape)} is not {(3, n) if three else (n,)}")
        if q is None and q_out is not None:
            raise PnbError(-1, "q_out: without q")
        if q is not None:
            q_out = self._rows(q if q_out is None else q_out, "q_out", n, self._n_head)
            q = self._rows(q, "q", n, self._n_head)
        check(pnb_pkv_append(self._h, _i32(layer, "layer"), self._batch(batch), n, self._rows(k, "k", n, self._n_kv),
                             self._rows(v, "v", n, self._n_kv), q, q_out,
                             None if pos is None else self._ints(pos, "pos"), self._stream(stream)),
              "pnb_pkv_append")

    def attention(self, layer: int, batch: PagedBatch, q, out, window: int = 0, stream=None):
        """Causal attention of the tokens' queries over their sequences' entries into ``out``."""
        n = _i32(q.shape[0], "tokens")
        check(pnb_pkv_attention(self._h, _i32(layer, "layer"), self._batch(batch), n,
                                self._rows(q, "q", n, self._n_head), self._rows(out, "out", n, self._n_head),
                                _i32(window, "window"), self._stream(stream)), "pnb_pkv_attention")

    def attention_shared(self, layer: int, batch: PagedBatch, group_start, prefix, q, out, window: int = 0,
                         stream=None):
        """The same for groups of sequences whose first ``prefix[g]`` entries lie in the same pages:
        group g is the sequences group_start[g] .. group_start[g + 1] - 1."""
        n, g = _i32(q.shape[0], "tokens"), prefix.numel()
        if prefix.shape != (g,) or group_start.shape != (g + 1,):
            raise PnbError(-1, f"group_start: shape {tuple(group_start.shape)} is not ({g + 1},)")
        check(pnb_pkv_attention_shared(self._h, _i32(layer, "layer"), self._batch(batch), g,
                                       self._ints(group_start, "group_start"), self._ints(prefix, "prefix"), n,
                                       self._rows(q, "q", n, self._n_head), self._rows(out, "out", n, self._n_head),
                                       _i32(window, "window"), self._stream(stream)), "pnb_pkv_attention_shared")

    def device_error(self) -> int:
        """Synchronise, read and clear the device error bits (PNB_DEV_ERR_*)."""
        e = ctypes.c_int32()
        rc = pnb_pkv_check(self._h, ctypes.byref(e))
        if rc not in (0, -8):
            check(rc, "pnb_pkv_check")
        return e.value
