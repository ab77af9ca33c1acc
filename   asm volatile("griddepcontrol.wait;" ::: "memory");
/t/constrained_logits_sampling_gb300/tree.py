"""The operators of a speculative step whose drafted tokens form a tree.

A request drafts several continuations of its last accepted token, the root: drafted token i
continues token ``parents[i]`` (-1: the root).  The step's rows are each request's root and then its
drafted tokens.  One step takes them through

* ``TreePlan``: what each row may see, its position and the rows' offsets, once for all layers;
* ``speculative.KVAppend`` with the plan's ``positions``, and ``TreeAttention`` with its ``mask``, in
  every layer;
* ``TreeVerifier``: a walk down the tree that accepts drafted tokens, and one more token per request;
* ``pages.KeepPath``: the accepted tokens' keys and values moved together, and the new lengths.

As in ``speculative``: argument marshalling only, ``make_args`` checks a call once, ``apply`` enqueues
it as often as wanted, calling an object does both and allocates the outputs.  The formulas and limits are
stated in include/clsample.h.
"""
from __future__ import annotations

import ctypes
from typing import Dict, Optional

import torch

from .sampler import LOGITS_BF16, LOGITS_F32, _check, _dptr, _stream_ptr, load_library
from .speculative import (_I32, _I64, _PTR, AttentionArgs, ChunkAttention, _Args, _current, _device, _on, _on_stream,
                          _writable)


class TreePlanArgs(_Args):
    """Mirror of clsample_tree_plan_args_t (include/clsample.h)."""
    _fields_ = [(n, _I32) for n in ("B", "N", "max_draft", "window")] + [
        (n, _PTR) for n in ("parents", "cu_draft", "kv_lens", "mask")] + [
        ("mask_stride", _I64), ("positions", _PTR), ("cu_new", _PTR), ("row_status", _PTR)]


class TreeMask(_Args):
    """Mirror of clsample_tree_mask_t (include/clsample.h)."""
    _fields_ = [("mask", _PTR), ("mask_stride", _I64), ("positions", _PTR)]


class VerifyTreeArgs(_Args):
    """Mirror of clsample_verify_tree_args_t (include/clsample.h)."""
    _fields_ = [(n, _I32) for n in ("B", "N", "V", "dtype", "max_draft", "max_path", "draft_rows_count", "reserved0")] + [
        ("target", _PTR), ("target_stride", _I64), ("draft", _PTR), ("draft_stride", _I64)] + [
        (n, _PTR) for n in ("draft_rows", "draft_tokens", "parents", "cu_draft", "u_accept", "u_sample", "tokens")] + [
        ("token_stride", _I64), ("path", _PTR), ("path_stride", _I64), ("accepted", _PTR), ("row_status", _PTR)]


def _row_stride(t: torch.Tensor, least: int) -> int:
    # a single row is never stepped over, whatever stride it carries
    return max(t.stride(0), least) if t.shape[0] <= 1 else t.stride(0)


class TreePlan:
    """Masks, positions and offsets of a batch of trees (``clsample_tree_plan``)."""

    def __init__(self):
        self._L = load_library()
        self.device = _device()

    def make_args(self, parents: torch.Tensor, cu_draft: torch.Tensor, kv_lens: torch.Tensor, *, max_draft: int,
                  window: int = 0, mask: torch.Tensor, positions: Optional[torch.Tensor] = None,
                  cu_new: Optional[torch.Tensor] = None, row_status: Optional[torch.Tensor] = None) -> TreePlanArgs:
        """parents int32 [N], cu_draft int32 [B + 1], kv_lens int32 [B] with the step's rows;
        ``max_draft``: no request has more drafted tokens; mask int32 [N + B, >= ceil((max_draft + 1) /
        32)], positions int32 [N + B], cu_new int32 [B + 1]."""
        dev = self.device
        a = TreePlanArgs()
        a.B, a.N, a.max_draft, a.window = kv_lens.numel(), parents.numel(), int(max_draft), int(window)
        a.parents = _dptr(parents, torch.int32, a.N, "parents", dev)
        a.cu_draft = _dptr(cu_draft, torch.int32, a.B + 1, "cu_draft", dev)
        a.kv_lens = _dptr(kv_lens, torch.int32, a.B, "kv_lens", dev)
        _on(mask, "mask", dev, torch.int32, 2)
        _writable(mask, "mask")
        words = (a.max_draft + 32) // 32
        if mask.shape[0] != a.N + a.B or mask.shape[1] < words:
            raise ValueError(f"mask has shape {tuple(mask.shape)}, expected [{a.N + a.B}, >= {words}]")
        a.mask, a.mask_stride = mask.data_ptr(), _row_stride(mask, words)
        a.positions = _dptr(positions, torch.int32, a.N + a.B, "positions", dev)
        a.cu_new = _dptr(cu_new, torch.int32, a.B + 1, "cu_new", dev)
        a.row_status = _dptr(row_status, torch.int32, a.B, "row_status", dev)
        a.keep = (parents, cu_draft, kv_lens, mask, positions, cu_new, row_status)
        return a

    def apply(self, args: TreePlanArgs, stream: Optional[torch.cuda.Stream] = None):
        """Enqueue one call on ``stream`` (default: current)."""
        _current(self.device)
        _check(self._L.clsample_tree_plan(ctypes.byref(args), _stream_ptr(stream)))

    def __call__(self, parents, cu_draft, kv_lens, *, max_draft: int, window: int = 0,
                 stream=None) -> Dict[str, torch.Tensor]:
        """Plan, and return ``mask`` int32 [N + B, words], ``positions`` int32 [N + B], ``cu_new`` int32
        [B + 1] and ``status`` (int32 per request)."""
        B, rows, dev = kv_lens.numel(), parents.numel() + kv_lens.numel(), parents.device
        with _on_stream(stream):
            # (zeros: rows of a request whose offsets are not in order are not written)
            out = {"mask": torch.zeros(rows, (int(max_draft) + 32) // 32, dtype=torch.int32, device=dev),
                   "positions": torch.zeros(rows, dtype=torch.int32, device=dev),
                   "cu_new": torch.empty(B + 1, dtype=torch.int32, device=dev),
                   "status": torch.empty(B, dtype=torch.int32, device=dev)}
            if B == 0:
                out["cu_new"].zero_()
        self.apply(self.make_args(parents, cu_draft, kv_lens, max_draft=max_draft, window=window, mask=out["mask"],
                                  positions=out["positions"], cu_new=out["cu_new"], row_status=out["status"]), stream)
        return out


class TreeAttention(ChunkAttention):
    """``ChunkAttention`` whose rows see their sequence's new tokens by mask
    (``clsample_tree_attention``)."""

    def make_args(self, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                  cu_new: torch.Tensor, kv_lens: torch.Tensor, *, mask: torch.Tensor,
                  positions: Optional[torch.Tensor] = None, max_new: Optional[int] = None, **kw) -> AttentionArgs:
        """As for ``ChunkAttention``.  mask int32 [T, words]: bit j & 31 of word j >> 5 of a row tells
        whether it sees its sequence's new token j; positions int32 [T] (None: places in the sequence) count
        for the window alone.  ``max_new`` None: as many as the mask has bits for."""
        dev = self.device
        _on(mask, "mask", dev, torch.int32, 2)
        T = q.shape[0]
        if mask.shape[0] != T:
            raise ValueError(f"mask has {mask.shape[0]} rows, expected {T}")
        if max_new is None:
            max_new = min(T, 32 * mask.shape[1])
        if int(max_new) > 32 * mask.shape[1]:
            raise ValueError(f"mask has {mask.shape[1]} words a row, max_new is {max_new}")
        a = super().make_args(q, k_cache, v_cache, page_table, cu_new, kv_lens, max_new=max_new, **kw)
        a.tree = TreeMask()
        a.tree.mask, a.tree.mask_stride = mask.data_ptr(), _row_stride(mask, mask.shape[1])
        a.tree.positions = _dptr(positions, torch.int32, T, "positions", dev)
        a.keep += (mask, positions)
        return a

    def apply(self, args: AttentionArgs, stream: Optional[torch.cuda.Stream] = None):
        """Enqueue one call on ``stream`` (default: current)."""
        _check(self._L.clsample_tree_attention(self._h, ctypes.byref(args), ctypes.byref(args.tree), _stream_ptr(stream)))


class TreeVerifier:
    """Acceptance of a path of drafted tokens and one more token per request
    (``clsample_verify_tree``)."""

    def __init__(self):
        self._L = load_library()
        self.device = _device()

    def make_args(self, target_probs: torch.Tensor, draft_tokens: torch.Tensor, parents: torch.Tensor,
                  cu_draft: torch.Tensor, u_accept: torch.Tensor, u_sample: torch.Tensor, *, max_draft: int,
                  max_path: Optional[int] = None, draft_probs: Optional[torch.Tensor] = None,
                  draft_rows: Optional[torch.Tensor] = None, tokens: torch.Tensor,
                  path: Optional[torch.Tensor] = None, accepted: Optional[torch.Tensor] = None,
                  row_status: Optional[torch.Tensor] = None) -> VerifyTreeArgs:
        """target_probs [N + B, V] (float32 or bfloat16) by rows of the step; draft_probs [M, V] of the
        same type, token i having been drawn from row draft_rows[i] (int32 [N]; None: row i), or None (a
        draft certain of its tokens); draft_tokens and parents int32 [N], cu_draft int32 [B + 1], u_accept
        float32 [N], u_sample float32 [B]; ``max_draft``: no request has more drafted tokens; ``max_path``
        (None: max_draft): no more are accepted; tokens int32 [B, > max_path], path int32 [B, >= max_path]."""
        dev, dt = self.device, target_probs.dtype
        a = VerifyTreeArgs()
        if dt == torch.float32:
            a.dtype = LOGITS_F32
        elif dt == torch.bfloat16:
            a.dtype = LOGITS_BF16
        else:
            raise ValueError(f"unsupported dtype {dt}")
        _on(target_probs, "target_probs", dev, dt, 2)
        a.B, a.N, a.V = u_sample.numel(), draft_tokens.numel(), target_probs.shape[1]
        if target_probs.shape[0] != a.N + a.B:
            raise ValueError(f"target_probs has {target_probs.shape[0]} rows, expected {a.N + a.B}")
        a.max_draft = int(max_draft)
        a.max_path = a.max_draft if max_path is None else int(max_path)
        a.target, a.target_stride = target_probs.data_ptr(), _row_stride(target_probs, a.V)
        if draft_probs is not None:
            _on(draft_probs, "draft_probs", dev, dt, 2)
            if draft_probs.shape[1] != a.V or (draft_rows is None and draft_probs.shape[0] != a.N):
                raise ValueError(f"draft_probs has shape {tuple(draft_probs.shape)}, expected "
                                 f"[{a.N if draft_rows is None else 'rows'}, {a.V}]")
            # without drafted tokens no draft row is ever read
            a.draft = draft_probs.data_ptr() if a.N else None
            if a.N and not a.draft:
                raise ValueError("draft_probs has no rows")
            a.draft_stride, a.draft_rows_count = _row_stride(draft_probs, a.V), draft_probs.shape[0]
        elif draft_rows is not None:
            raise ValueError("draft_rows needs draft_probs")
        a.draft_rows = _dptr(draft_rows, torch.int32, a.N, "draft_rows", dev)
        a.draft_tokens = _dptr(draft_tokens, torch.int32, a.N, "draft_tokens", dev)
        a.parents = _dptr(parents, torch.int32, a.N, "parents", dev)
        a.cu_draft = _dptr(cu_draft, torch.int32, a.B + 1, "cu_draft", dev)
        a.u_accept = _dptr(u_accept, torch.float32, a.N, "u_accept", dev)
        a.u_sample = _dptr(u_sample, torch.float32, a.B, "u_sample", dev)
        _on(tokens, "tokens", dev, torch.int32, 2)
        if tokens.shape[0] != a.B or tokens.shape[1] <= a.max_path:
            raise ValueError(f"tokens has shape {tuple(tokens.shape)}, expected [{a.B}, > {a.max_path}]")
        _writable(tokens, "tokens")
        a.tokens, a.token_stride = tokens.data_ptr(), _row_stride(tokens, a.max_path + 1)
        if path is not None:
            _on(path, "path", dev, torch.int32, 2)
            if path.shape[0] != a.B or path.shape[1] < a.max_path:
                raise ValueError(f"path has shape {tuple(path.shape)}, expected [{a.B}, >= {a.max_path}]")
            _writable(path, "path")
            a.path, a.path_stride = path.data_ptr(), _row_stride(path, a.max_path)
        a.accepted = _dptr(accepted, torch.int32, a.B, "accepted", dev)
        a.row_status = _dptr(row_status, torch.int32, a.B, "row_status", dev)
        a.keep = (target_probs, draft_probs, draft_rows, draft_tokens, parents, cu_draft, u_accept, u_sample, tokens,
                  path, accepted, row_status)
        return a

    def apply(self, args: VerifyTreeArgs, stream: Optional[torch.cuda.Stream] = None):
        """Enqueue one call on ``stream`` (default: current)."""
        _current(self.device)
        _check(self._L.clsample_verify_tree(ctypes.byref(args), _stream_ptr(stream)))

    def __call__(self, target_probs, draft_tokens, parents, cu_draft, u_accept, u_sample, *, max_draft: int,
                 max_path: Optional[int] = None, draft_probs=None, draft_rows=None,
                 stream=None) -> Dict[str, torch.Tensor]:
        """Verify, and return ``tokens`` int32 [B, max_path + 1] (accepted tokens, the drawn token, then
        -1), ``path`` int32 [B, max_path] (the accepted tokens' numbers, then -1), ``accepted`` and
        ``status`` (int32 per request)."""
        B, dev = u_sample.numel(), target_probs.device
        most = int(max_draft) if max_path is None else int(max_path)
        with _on_stream(stream):
            out = {"tokens": torch.empty(B, most + 1, dtype=torch.int32, device=dev),
                   "path": torch.empty(B, most, dtype=torch.int32, device=dev),
                   "accepted": torch.empty(B, dtype=torch.int32, device=dev),
                   "status": torch.empty(B, dtype=torch.int32, device=dev)}
        self.apply(self.make_args(target_probs, draft_tokens, parents, cu_draft, u_accept, u_sample,
                                  max_draft=max_draft, max_path=most, draft_probs=draft_probs, draft_rows=draft_rows,
                                  tokens=out["tokens"], path=out["path"], accepted=out["accepted"],
                                  row_status=out["status"]), stream)
        return out
