"""Pages of a cache: which sequence holds which, and keys and values moved between them.

* ``PagePool``: pages that sequences may share, counted on the device.  ``fork`` makes a sequence a
  copy of another that shares its pages, ``reserve`` gives sequences the pages that their next tokens
  need (and one of their own for each shared page that they would write to), ``trim`` takes back what
  a sequence's length no longer needs.
* ``CopyPages``: the tokens of pages that ``reserve`` replaced, copied in all layers.
* ``KeepPath``: keys and values of the accepted path of a tree of drafted tokens moved together in all
  layers, and the new lengths.

A batch has ``page_table`` int32 [B, max_pages] as the attention reads it, ``held`` int32 [B] (how many
entries of its row a sequence holds) and ``kv_lens`` int32 [B]; all start as zeros.  Caches are [pages, page_size,
Hkv, D] or [layers, pages, page_size, Hkv, D] with any strides.

As in ``speculative``: argument marshalling only, ``*_args`` check a call once, ``apply`` enqueues it as often as
wanted, the other calls do both and allocate the outputs.  The rules are stated in include/clsample.h.
"""
from __future__ import annotations

import ctypes
from typing import Dict, Optional

import torch

from .sampler import _check, _dptr, _stream_ptr, load_library
from .speculative import _I32, _I64, _PTR, _Args, _current, _device, _on, _on_stream, _stride, _type_of, _writable
from .tree import _row_stride


class KeepPathArgs(_Args):
    """Mirror of clsample_keep_path_args_t (include/clsample.h)."""
    _fields_ = [(n, _I32) for n in ("B", "N", "layers", "Hkv", "D", "dtype", "num_pages", "page_size", "max_pages",
                                    "max_path")] + [
        ("k_cache", _PTR), ("v_cache", _PTR)] + [
        (n, _I64) for n in ("layer_stride", "page_stride", "slot_stride", "head_stride")] + [
        ("page_table", _PTR), ("table_stride", _I64), ("cu_draft", _PTR), ("kv_lens", _PTR), ("path", _PTR),
        ("path_stride", _I64), ("accepted", _PTR), ("new_lens", _PTR), ("row_status", _PTR)]


class CopyPagesArgs(_Args):
    """Mirror of clsample_copy_pages_args_t (include/clsample.h)."""
    _fields_ = [(n, _I32) for n in ("n", "layers", "Hkv", "D", "dtype", "num_pages", "page_size", "reserved0")] + [
        ("k_cache", _PTR), ("v_cache", _PTR)] + [
        (n, _I64) for n in ("layer_stride", "page_stride", "slot_stride", "head_stride")] + [
        ("copies", _PTR), ("status", _PTR)]


class PoolArgs(_Args):
    """Mirror of clsample_page_pool_t (include/clsample.h)."""
    _fields_ = [("num_pages", _I32), ("page_size", _I32)] + [
        (n, _PTR) for n in ("refs", "free_bits", "stamps", "epoch", "list")]


class BatchArgs(_Args):
    """Mirror of clsample_page_batch_t (include/clsample.h)."""
    _fields_ = [("B", _I32), ("max_pages", _I32), ("page_table", _PTR), ("table_stride", _I64), ("held", _PTR),
                ("kv_lens", _PTR)]


def _set_layers(a, k_cache, v_cache, dev):
    """The cache's fields, of a cache with or without a dimension of layers."""
    if k_cache.dim() not in (4, 5):
        raise ValueError("k_cache must be [pages, page_size, Hkv, D] or [layers, pages, page_size, Hkv, D]")
    a.dtype = _type_of(k_cache)
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _on(t, name, dev, k_cache.dtype, k_cache.dim())
        _writable(t, name)
    if k_cache.dim() == 4:
        k_cache, v_cache = k_cache.unsqueeze(0), v_cache.unsqueeze(0)
    if k_cache.shape != v_cache.shape or any(_stride(k_cache, i) != _stride(v_cache, i) for i in range(4)):
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    a.layers, a.num_pages, a.page_size, a.Hkv, a.D = k_cache.shape
    a.k_cache, a.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
    a.layer_stride, a.page_stride, a.slot_stride, a.head_stride = (_stride(k_cache, i) for i in range(4))


class KeepPath:
    """Accepted paths of trees of drafted tokens moved together (``clsample_keep_path``)."""

    def __init__(self):
        self._L = load_library()
        self.device = _device()

    def make_args(self, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, cu_draft: torch.Tensor,
                  kv_lens: torch.Tensor, path: torch.Tensor, accepted: torch.Tensor, *, new_lens: torch.Tensor,
                  row_status: Optional[torch.Tensor] = None) -> KeepPathArgs:
        """cu_draft int32 [B + 1], kv_lens int32 [B] with the step's rows, path int32 [B, max_path] and
        accepted int32 [B] as ``tree.TreeVerifier`` leaves them; new_lens int32 [B], another tensor than
        kv_lens."""
        dev = self.device
        a = KeepPathArgs()
        _set_layers(a, k_cache, v_cache, dev)
        a.B = kv_lens.numel()
        _on(page_table, "page_table", dev, torch.int32, 2)
        _on(path, "path", dev, torch.int32, 2)
        if page_table.shape[0] != a.B or path.shape[0] != a.B:
            raise ValueError(f"page_table and path have {page_table.shape[0]} and {path.shape[0]} rows, expected {a.B}")
        a.max_pages, a.max_path = page_table.shape[1], path.shape[1]
        a.page_table, a.table_stride = page_table.data_ptr(), _row_stride(page_table, a.max_pages)
        a.path, a.path_stride = path.data_ptr(), _row_stride(path, a.max_path)
        a.N = (1 << 31) - 1  # no token array to stay within
        a.cu_draft = _dptr(cu_draft, torch.int32, a.B + 1, "cu_draft", dev)
        a.kv_lens = _dptr(kv_lens, torch.int32, a.B, "kv_lens", dev)
        a.accepted = _dptr(accepted, torch.int32, a.B, "accepted", dev)
        a.new_lens = _dptr(new_lens, torch.int32, a.B, "new_lens", dev)
        a.row_status = _dptr(row_status, torch.int32, a.B, "row_status", dev)
        a.keep = (k_cache, v_cache, page_table, cu_draft, kv_lens, path, accepted, new_lens, row_status)
        return a

    def apply(self, args: KeepPathArgs, stream: Optional[torch.cuda.Stream] = None):
        """Enqueue one call on ``stream`` (default: current)."""
        _current(self.device)
        _check(self._L.clsample_keep_path(ctypes.byref(args), _stream_ptr(stream)))

    def __call__(self, k_cache, v_cache, page_table, cu_draft, kv_lens, path, accepted, *,
                 stream=None) -> Dict[str, torch.Tensor]:
        """Move, and return ``kv_lens`` (the new lengths) and ``status`` (int32 per sequence)."""
        with _on_stream(stream):
            out = {n: torch.empty(kv_lens.numel(), dtype=torch.int32, device=kv_lens.device) for n in ("kv_lens", "status")}
        self.apply(self.make_args(k_cache, v_cache, page_table, cu_draft, kv_lens, path, accepted,
                                  new_lens=out["kv_lens"], row_status=out["status"]), stream)
        return out


class CopyPages:
    """First slots of pages copied to other pages in all layers (``clsample_copy_pages``)."""

    def __init__(self):
        self._L = load_library()
        self.device = _device()

    def make_args(self, k_cache: torch.Tensor, v_cache: torch.Tensor, copies: torch.Tensor, *,
                  status: Optional[torch.Tensor] = None) -> CopyPagesArgs:
        """copies int32 [n, 3]: (from, to, slots), as ``PagePool.reserve`` gives them; from < 0: none."""
        dev = self.device
        a = CopyPagesArgs()
        _set_layers(a, k_cache, v_cache, dev)
        if copies.dim() != 2 or copies.shape[1] != 3:
            raise ValueError(f"copies has shape {tuple(copies.shape)}, expected [n, 3]")
        a.n = copies.shape[0]
        a.copies = _dptr(copies, torch.int32, 3 * a.n, "copies", dev)
        a.status = _dptr(status, torch.int32, a.n, "status", dev)
        a.keep = (k_cache, v_cache, copies, status)
        return a

    def apply(self, args: CopyPagesArgs, stream: Optional[torch.cuda.Stream] = None):
        """Enqueue one call on ``stream`` (default: current)."""
        _current(self.device)
        _check(self._L.clsample_copy_pages(ctypes.byref(args), _stream_ptr(stream)))

    def __call__(self, k_cache, v_cache, copies, *, stream=None) -> torch.Tensor:
        """Copy, and return a status per copy (int32)."""
        with _on_stream(stream):
            status = torch.empty(copies.shape[0], dtype=torch.int32, device=copies.device)
        self.apply(self.make_args(k_cache, v_cache, copies, status=status), stream)
        return status


class _PoolCall:
    """A checked call of a pool: the name of the library's function, its arguments, and what it keeps alive (the
    pool among it)."""

    def __init__(self, name, pool, batch, args, keep):
        self.name, self.keep = name, (pool, batch, keep)
        self.args = (ctypes.byref(pool), ctypes.byref(batch)) + args


class PagePool:
    """``num_pages`` pages of ``page_size`` slots on the current device, all of them free.  ``refs`` int32
    [num_pages] tells how many sequences hold a page.  Calls on one pool, ``load`` among them, have to be ordered;
    a new pool is ready for any stream (making one waits for the current stream, except while a graph is captured:
    such a pool starts anew with each replay, on the capture's streams)."""

    def __init__(self, num_pages: int, page_size: int):
        self._L = load_library()
        self.device = _device()
        self.num_pages, self.page_size = int(num_pages), int(page_size)
        if self.num_pages < 0 or self.page_size < 1:
            raise ValueError(f"a pool of {num_pages} pages of {page_size} slots")
        n, dev = self.num_pages, self.device
        self.refs = torch.zeros(n, dtype=torch.int32, device=dev)
        self.free_bits = torch.empty((n + 31) // 32, dtype=torch.int32, device=dev)
        self._stamps = torch.zeros(n, dtype=torch.int64, device=dev)
        self._epoch = torch.zeros(1, dtype=torch.int32, device=dev)
        self._list = torch.zeros(n, dtype=torch.int32, device=dev)
        p = self._args = PoolArgs()
        p.num_pages, p.page_size = n, self.page_size
        p.refs, p.free_bits, p.stamps = self.refs.data_ptr(), self.free_bits.data_ptr(), self._stamps.data_ptr()
        p.epoch, p.list = self._epoch.data_ptr(), self._list.data_ptr()
        self._set_free()
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.device).synchronize()

    def _set_free(self):
        free = torch.zeros(32 * self.free_bits.numel(), dtype=torch.int64, device=self.device)
        free[:self.num_pages] = (self.refs == 0).long()
        bits = (free.view(-1, 32) << torch.arange(32, device=self.device)).sum(1)
        self.free_bits.copy_(torch.where(bits >= 1 << 31, bits - (1 << 32), bits))

    def load(self, refs: torch.Tensor, stream: Optional[torch.cuda.Stream] = None):
        """Start from other counts of holders (int32 [num_pages]), those of tables made elsewhere.  Enqueued on
        ``stream`` (default: current)."""
        if refs.dtype != torch.int32 or tuple(refs.shape) != (self.num_pages,):
            raise ValueError(f"refs must be int32 [{self.num_pages}]")
        with _on_stream(stream):
            self.refs.copy_(refs)
            self._set_free()

    def _batch(self, page_table, held, kv_lens):
        b, dev = BatchArgs(), self.device
        b.B = held.numel()
        _on(page_table, "page_table", dev, torch.int32, 2)
        _writable(page_table, "page_table")
        if page_table.shape[0] != b.B:
            raise ValueError(f"page_table has {page_table.shape[0]} rows, expected {b.B}")
        b.max_pages = page_table.shape[1]
        b.page_table, b.table_stride = page_table.data_ptr(), _row_stride(page_table, b.max_pages)
        b.held = _dptr(held, torch.int32, b.B, "held", dev)
        b.kv_lens = _dptr(kv_lens, torch.int32, b.B, "kv_lens", dev)
        return b

    def fork_args(self, page_table: torch.Tensor, held: torch.Tensor, kv_lens: torch.Tensor, src: torch.Tensor,
                  dst: torch.Tensor, *, row_status: Optional[torch.Tensor] = None) -> _PoolCall:
        """src and dst int32 [n]: sequence dst[i], which holds nothing, becomes a copy of src[i]."""
        dev, n = self.device, src.numel()
        b = self._batch(page_table, held, kv_lens)
        args = (_dptr(src, torch.int32, n, "src", dev), _dptr(dst, torch.int32, n, "dst", dev), n,
                _dptr(row_status, torch.int32, n, "row_status", dev))
        return _PoolCall("clsample_pages_fork", self._args, b, args,
                         (self, page_table, held, kv_lens, src, dst, row_status))

    def reserve_args(self, page_table: torch.Tensor, held: torch.Tensor, kv_lens: torch.Tensor,
                     new_tokens: torch.Tensor, *, copies: torch.Tensor, row_status: Optional[torch.Tensor] = None,
                     free_pages: Optional[torch.Tensor] = None) -> _PoolCall:
        """new_tokens int32 [B]: how many tokens each sequence is to write behind kv_lens; copies int32
        [B, 3], free_pages int32 [1] (left after the call)."""
        dev = self.device
        b = self._batch(page_table, held, kv_lens)
        args = (_dptr(new_tokens, torch.int32, b.B, "new_tokens", dev), _dptr(copies, torch.int32, 3 * b.B, "copies", dev),
                _dptr(row_status, torch.int32, b.B, "row_status", dev),
                _dptr(free_pages, torch.int32, 1, "free_pages", dev))
        return _PoolCall("clsample_pages_reserve", self._args, b, args,
                         (self, page_table, held, kv_lens, new_tokens, copies, row_status, free_pages))

    def trim_args(self, page_table: torch.Tensor, held: torch.Tensor, kv_lens: torch.Tensor, *,
                  row_status: Optional[torch.Tensor] = None) -> _PoolCall:
        """Each sequence keeps the pages that kv_lens needs."""
        b = self._batch(page_table, held, kv_lens)
        args = (_dptr(row_status, torch.int32, b.B, "row_status", self.device),)
        return _PoolCall("clsample_pages_trim", self._args, b, args, (self, page_table, held, kv_lens, row_status))

    def apply(self, call: _PoolCall, stream: Optional[torch.cuda.Stream] = None):
        """Enqueue one call on ``stream`` (default: current)."""
        _current(self.device)
        _check(getattr(self._L, call.name)(*call.args, _stream_ptr(stream)))

    def _new(self, stream, *shapes):
        with _on_stream(stream):
            return [torch.empty(s, dtype=torch.int32, device=self.device) for s in shapes]

    def fork(self, page_table, held, kv_lens, src, dst, *, stream=None) -> torch.Tensor:
        """Fork, and return a status per pair (int32)."""
        status, = self._new(stream, (src.numel(),))
        self.apply(self.fork_args(page_table, held, kv_lens, src, dst, row_status=status), stream)
        return status

    def reserve(self, page_table, held, kv_lens, new_tokens, *, stream=None) -> Dict[str, torch.Tensor]:
        """Reserve, and return ``copies`` int32 [B, 3] (for ``CopyPages``, before the tokens are written),
        ``free`` int32 [1] (pages left) and ``status`` (int32 per sequence)."""
        B = held.numel()
        copies, free, status = self._new(stream, (B, 3), (1,), (B,))
        self.apply(self.reserve_args(page_table, held, kv_lens, new_tokens, copies=copies, row_status=status,
                                     free_pages=free), stream)
        return {"copies": copies, "free": free, "status": status}

    def trim(self, page_table, held, kv_lens, *, stream=None) -> torch.Tensor:
        """Trim, and return a status per sequence (int32)."""
        status, = self._new(stream, (held.numel(),))
        self.apply(self.trim_args(page_table, held, kv_lens, row_status=status), stream)
        return status
