"""The other operators of a speculative-decoding step, next to the sampler.

One step takes the newest tokens of each sequence (one token, the last accepted token and
the drafted ones, or a chunk of a prompt) through

* ``KVAppend``: norm of queries and keys per head, position rotation, keys and values into
  a paged cache;
* ``ChunkAttention``: attention of those tokens over the cache;
* ``DraftVerifier``: drafted tokens accepted against the target's probabilities, and one
  more token per request, from given random numbers.

As in ``sampler``, this is argument marshalling only: every step runs in libclsample.so, on
CUDA tensors, without a CPU fallback.  ``make_args`` checks a call once and keeps its
tensors alive, and the object whose scratch it takes (a captured graph needs them for as long as it is
replayed); ``apply`` enqueues it, as often as wanted (the buffers' contents may change
in between).  Calling an object does both and allocates the outputs.  An object belongs to the
device that was current when it was made, and refuses calls while another one is.  The
formulas and limits are stated in include/clsample.h.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Dict, Optional

import torch

from .sampler import LOGITS_BF16, LOGITS_F32, ClsampleError, _check, _dptr, _stream_ptr, load_library

T_BF16, T_F16 = 0, 1
ERR_DEVICE = -7
_I32, _I64, _PTR = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class _Args(ctypes.Structure):
    """Numbers that a 32-bit field cannot hold are refused: ctypes would keep their low bits."""

    def __init_subclass__(cls):
        cls._narrow = frozenset(n for n, t in cls._fields_ if t is _I32)

    def __setattr__(self, name, value):
        if name in self._narrow and not -(1 << 31) <= value < 1 << 31:
            raise ValueError(f"{name} is {value}: out of the 32-bit range")
        super().__setattr__(name, value)


class KVAppendArgs(_Args):
    """Mirror of clsample_kv_append_args_t (include/clsample.h)."""
    _fields_ = [(n, _I32) for n in ("B", "T", "Hq", "Hkv", "D", "dtype", "num_pages", "page_size", "max_pages",
                                    "rot_dim", "max_pos", "interleaved")] + [
        ("eps", ctypes.c_float), ("reserved0", _I32)] + [
        (n, _PTR) for n in ("q", "k", "v", "q_out", "k_cache", "v_cache")] + [
        (n, _I64) for n in ("q_stride_t", "q_stride_h", "k_stride_t", "k_stride_h", "v_stride_t", "v_stride_h",
                            "qo_stride_t", "qo_stride_h", "page_stride", "slot_stride", "head_stride")] + [
        ("page_table", _PTR), ("table_stride", _I64), ("cu_new", _PTR), ("kv_lens", _PTR), ("cos_sin", _PTR),
        ("cs_stride", _I64), ("q_weight", _PTR), ("k_weight", _PTR), ("row_status", _PTR)]


class AttentionArgs(_Args):
    """Mirror of clsample_attention_args_t (include/clsample.h)."""
    _fields_ = [(n, _I32) for n in ("B", "T", "Hq", "Hkv", "D", "dtype", "num_pages", "page_size", "max_pages",
                                    "max_new", "window")] + [("scale", ctypes.c_float)] + [
        (n, _PTR) for n in ("q", "out", "k_cache", "v_cache")] + [
        (n, _I64) for n in ("q_stride_t", "q_stride_h", "o_stride_t", "o_stride_h", "page_stride", "slot_stride",
                            "head_stride")] + [
        ("page_table", _PTR), ("table_stride", _I64), ("cu_new", _PTR), ("kv_lens", _PTR), ("lse", _PTR),
        ("row_status", _PTR)]


class VerifyArgs(_Args):
    """Mirror of clsample_verify_args_t (include/clsample.h)."""
    _fields_ = [(n, _I32) for n in ("B", "N", "V", "dtype", "max_draft", "reserved0")] + [
        ("target", _PTR), ("target_stride", _I64), ("draft", _PTR), ("draft_stride", _I64), ("draft_tokens", _PTR),
        ("cu_draft", _PTR), ("u_accept", _PTR), ("u_sample", _PTR), ("tokens", _PTR), ("token_stride", _I64),
        ("accepted", _PTR), ("row_status", _PTR)]


def _device() -> torch.device:
    if not torch.cuda.is_available():
        raise RuntimeError("the operators need a CUDA device")
    return torch.device("cuda", torch.cuda.current_device())


def _current(device: torch.device):
    # without a handle the library cannot know whose tensors a call has
    if torch.cuda.current_device() != device.index:
        raise ClsampleError(ERR_DEVICE)


def _on_stream(stream):
    # outputs belong to the stream that writes them
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _on(t: torch.Tensor, name: str, device: torch.device, dtype, dims: int):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != dims or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must have {dims} dimensions and unit stride in the last")


def _stride(t: torch.Tensor, i: int) -> int:
    # a dimension of one element is never stepped over, whatever stride it carries
    return t.stride(i) if t.shape[i] > 1 else 0


def _writable(t: torch.Tensor, name: str):
    if any(t.shape[i] > 1 and t.stride(i) == 0 for i in range(t.dim())):
        raise ValueError(f"{name} is written: it must not be expanded")


def _type_of(q: torch.Tensor) -> int:
    if q.dtype == torch.bfloat16:
        return T_BF16
    if q.dtype == torch.float16:
        return T_F16
    raise ValueError(f"unsupported dtype {q.dtype}")


def _set_cache(a, k_cache, v_cache, page_table, cu_new, kv_lens, dtype, dev):
    """The cache and batch fields that append and attention share."""
    _on(k_cache, "k_cache", dev, dtype, 4)
    _on(v_cache, "v_cache", dev, dtype, 4)
    if k_cache.shape != v_cache.shape or any(_stride(k_cache, i) != _stride(v_cache, i) for i in range(3)):
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    _on(page_table, "page_table", dev, torch.int32, 2)
    a.B = kv_lens.numel()
    if page_table.shape[0] != a.B:
        raise ValueError(f"page_table has {page_table.shape[0]} rows, expected {a.B}")
    a.num_pages, a.page_size, a.Hkv, a.D = k_cache.shape
    a.max_pages = page_table.shape[1]
    a.k_cache, a.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
    a.page_stride, a.slot_stride, a.head_stride = (_stride(k_cache, i) for i in range(3))
    a.page_table = page_table.data_ptr()
    a.table_stride = max(page_table.stride(0), a.max_pages) if a.B <= 1 else page_table.stride(0)
    a.cu_new = _dptr(cu_new, torch.int32, a.B + 1, "cu_new", dev)
    a.kv_lens = _dptr(kv_lens, torch.int32, a.B, "kv_lens", dev)


def _rows(t, name, dev, dtype, T, H, D):
    _on(t, name, dev, dtype, 3)
    if tuple(t.shape) != (T, H, D):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(T, H, D)}")
    return t.data_ptr(), _stride(t, 0), _stride(t, 1)


class KVAppend:
    """Norm, rotation and append to a paged cache (``clsample_kv_append``)."""

    def __init__(self):
        self._L = load_library()
        self.device = _device()

    def make_args(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                  v_cache: torch.Tensor, page_table: torch.Tensor, cu_new: torch.Tensor, kv_lens: torch.Tensor, *,
                  cos_sin: Optional[torch.Tensor] = None, rot_dim: Optional[int] = None, interleaved: bool = False,
                  q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                  eps: float = 1e-6, q_out: Optional[torch.Tensor] = None,
                  row_status: Optional[torch.Tensor] = None,
                  positions: Optional[torch.Tensor] = None) -> KVAppendArgs:
        """q [T, Hq, D], k and v [T, Hkv, D]; caches [pages, page_size, Hkv, D] (any strides, so
        a transposed view of another layout will do); page_table int32 [B, max_pages], cu_new
        int32 [B + 1], kv_lens int32 [B] with the new tokens.  ``cos_sin`` float32 [positions,
        rot_dim], cosines then sines; None: no rotation.  ``q_out`` None: q in place.  ``positions``
        int32 [T]: what each token is rotated by, where that is not its place in the sequence (a tree of
        drafted tokens, ``tree.TreePlan``)."""
        dev, dt = self.device, k.dtype
        a = KVAppendArgs()
        a.dtype = _type_of(k)
        _set_cache(a, k_cache, v_cache, page_table, cu_new, kv_lens, dt, dev)
        _writable(k_cache, "k_cache")
        _writable(v_cache, "v_cache")
        if q.dim() != 3:
            raise ValueError("q must be [T, Hq, D]")
        a.T, a.Hq = q.shape[0], q.shape[1]
        q_out = q if q_out is None else q_out
        a.q, a.q_stride_t, a.q_stride_h = _rows(q, "q", dev, dt, a.T, a.Hq, a.D)
        a.k, a.k_stride_t, a.k_stride_h = _rows(k, "k", dev, dt, a.T, a.Hkv, a.D)
        a.v, a.v_stride_t, a.v_stride_h = _rows(v, "v", dev, dt, a.T, a.Hkv, a.D)
        a.q_out, a.qo_stride_t, a.qo_stride_h = _rows(q_out, "q_out", dev, dt, a.T, a.Hq, a.D)
        _writable(q_out, "q_out")
        if cos_sin is not None:
            _on(cos_sin, "cos_sin", dev, torch.float32, 2)
            a.max_pos, a.rot_dim = cos_sin.shape[0], cos_sin.shape[1] if rot_dim is None else int(rot_dim)
            if a.rot_dim > cos_sin.shape[1]:
                raise ValueError(f"cos_sin has {cos_sin.shape[1]} columns, rot_dim is {a.rot_dim}")
            a.cos_sin = cos_sin.data_ptr()
            a.cs_stride = max(cos_sin.stride(0), a.rot_dim) if a.max_pos <= 1 else cos_sin.stride(0)
        elif rot_dim:
            raise ValueError("rot_dim needs cos_sin")
        a.interleaved, a.eps = int(interleaved), float(eps)
        a.q_weight = _dptr(q_weight, dt, a.D, "q_weight", dev)
        a.k_weight = _dptr(k_weight, dt, a.D, "k_weight", dev)
        a.row_status = _dptr(row_status, torch.int32, a.B, "row_status", dev)
        a.positions = _dptr(positions, torch.int32, a.T, "positions", dev)
        a.keep = (q, k, v, k_cache, v_cache, page_table, cu_new, kv_lens, cos_sin, q_weight, k_weight, q_out,
                  row_status, positions)
        return a

    def apply(self, args: KVAppendArgs, stream: Optional[torch.cuda.Stream] = None):
        """Enqueue one call on ``stream`` (default: current)."""
        _current(self.device)
        positions = getattr(args, "positions", None)
        if positions is None:
            _check(self._L.clsample_kv_append(ctypes.byref(args), _stream_ptr(stream)))
        else:
            _check(self._L.clsample_kv_append_at(ctypes.byref(args), positions, _stream_ptr(stream)))

    def __call__(self, q, k, v, k_cache, v_cache, page_table, cu_new, kv_lens, *, stream=None,
                 **kw) -> Dict[str, torch.Tensor]:
        """Append, and return ``q`` (normed and rotated, a new tensor unless ``q_out`` is
        given) and ``status`` (int32 per sequence)."""
        with _on_stream(stream):
            if kw.get("q_out") is None:
                kw["q_out"] = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if kw.get("row_status") is None:
                kw["row_status"] = torch.empty(kv_lens.numel(), dtype=torch.int32, device=q.device)
        self.apply(self.make_args(q, k, v, k_cache, v_cache, page_table, cu_new, kv_lens, **kw), stream)
        return {"q": kw["q_out"], "status": kw["row_status"]}


class ChunkAttention:
    """Attention of each sequence's newest tokens over its paged cache, on the current
    device (``clsample_chunk_attention``).  Holds the scratch in which the parts of a split
    key axis meet, so calls on one object must be ordered."""

    def __init__(self):
        self._L = load_library()
        self.device = _device()
        h = ctypes.c_void_p()
        _check(self._L.clsample_attention_create(ctypes.byref(h)))
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            self._L.clsample_attention_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def make_args(self, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                  cu_new: torch.Tensor, kv_lens: torch.Tensor, *, max_new: Optional[int] = None,
                  scale: Optional[float] = None, window: int = 0, out: torch.Tensor,
                  lse: Optional[torch.Tensor] = None, row_status: Optional[torch.Tensor] = None) -> AttentionArgs:
        """q and out [T, Hq, D]; the cache and batch as in ``KVAppend``.  ``max_new``: no
        sequence has more new tokens (None: T, a loose bound for a batch: with a bound of up to 16
        packed rows, max_new Hq / Hkv, the kernel for few rows runs alone); ``scale`` None:
        1 / sqrt(D); ``window`` > 0: a token sees only that many keys, itself included; ``lse``
        float32 [T, Hq]."""
        dev, dt = self.device, q.dtype
        a = AttentionArgs()
        a.dtype = _type_of(q)
        _set_cache(a, k_cache, v_cache, page_table, cu_new, kv_lens, dt, dev)
        if q.dim() != 3:
            raise ValueError("q must be [T, Hq, D]")
        a.T, a.Hq = q.shape[0], q.shape[1]
        a.q, a.q_stride_t, a.q_stride_h = _rows(q, "q", dev, dt, a.T, a.Hq, a.D)
        a.out, a.o_stride_t, a.o_stride_h = _rows(out, "out", dev, dt, a.T, a.Hq, a.D)
        _writable(out, "out")
        a.max_new = a.T if max_new is None else int(max_new)
        a.window = int(window)
        a.scale = 1.0 / math.sqrt(max(a.D, 1)) if scale is None else float(scale)
        a.lse = _dptr(lse, torch.float32, a.T * a.Hq, "lse", dev)
        a.row_status = _dptr(row_status, torch.int32, a.B, "row_status", dev)
        a.keep = (q, k_cache, v_cache, page_table, cu_new, kv_lens, out, lse, row_status, self)  # self: the scratch
        return a

    def apply(self, args: AttentionArgs, stream: Optional[torch.cuda.Stream] = None):
        """Enqueue one call on ``stream`` (default: current)."""
        _check(self._L.clsample_chunk_attention(self._h, ctypes.byref(args), _stream_ptr(stream)))

    def __call__(self, q, k_cache, v_cache, page_table, cu_new, kv_lens, *, lse: bool = False, stream=None,
                 **kw) -> Dict[str, torch.Tensor]:
        """Attend, and return ``out`` [T, Hq, D], ``status`` (int32 per sequence) and, with
        ``lse``, ``lse`` [T, Hq] (float32).  Rows that no sequence owns are not written."""
        with _on_stream(stream):
            if kw.get("out") is None:
                kw["out"] = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if kw.get("row_status") is None:
                kw["row_status"] = torch.empty(kv_lens.numel(), dtype=torch.int32, device=q.device)
            sums = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if lse else None
        self.apply(self.make_args(q, k_cache, v_cache, page_table, cu_new, kv_lens, lse=sums, **kw), stream)
        out = {"out": kw["out"], "status": kw["row_status"]}
        if lse:
            out["lse"] = sums
        return out


class DraftVerifier:
    """Acceptance of drafted tokens and one more token per request (``clsample_verify``)."""

    def __init__(self):
        self._L = load_library()
        self.device = _device()

    def make_args(self, target_probs: torch.Tensor, draft_tokens: torch.Tensor, cu_draft: torch.Tensor,
                  u_accept: torch.Tensor, u_sample: torch.Tensor, *, max_draft: int,
                  draft_probs: Optional[torch.Tensor] = None, tokens: torch.Tensor,
                  accepted: Optional[torch.Tensor] = None,
                  row_status: Optional[torch.Tensor] = None) -> VerifyArgs:
        """target_probs [N + B, V] (float32 or bfloat16; request b's rows start at
        cu_draft[b] + b), draft_probs [N, V] of the same type or None (a draft certain of its
        tokens), draft_tokens int32 [N], cu_draft int32 [B + 1], u_accept float32 [N], u_sample
        float32 [B]; ``max_draft``: no request has more drafted tokens; tokens int32
        [B, > max_draft]."""
        dev, dt = self.device, target_probs.dtype
        a = VerifyArgs()
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
        a.target = target_probs.data_ptr()
        a.target_stride = max(target_probs.stride(0), a.V) if a.N + a.B <= 1 else target_probs.stride(0)
        if draft_probs is not None:
            _on(draft_probs, "draft_probs", dev, dt, 2)
            if tuple(draft_probs.shape) != (a.N, a.V):
                raise ValueError(f"draft_probs has shape {tuple(draft_probs.shape)}, expected {(a.N, a.V)}")
            # without drafted tokens no draft row is ever read
            a.draft = draft_probs.data_ptr() if a.N else None
            a.draft_stride = max(draft_probs.stride(0), a.V) if a.N <= 1 else draft_probs.stride(0)
        a.draft_tokens = _dptr(draft_tokens, torch.int32, a.N, "draft_tokens", dev)
        a.cu_draft = _dptr(cu_draft, torch.int32, a.B + 1, "cu_draft", dev)
        a.u_accept = _dptr(u_accept, torch.float32, a.N, "u_accept", dev)
        a.u_sample = _dptr(u_sample, torch.float32, a.B, "u_sample", dev)
        _on(tokens, "tokens", dev, torch.int32, 2)
        if tokens.shape[0] != a.B or tokens.shape[1] <= a.max_draft:
            raise ValueError(f"tokens has shape {tuple(tokens.shape)}, expected [{a.B}, > {a.max_draft}]")
        _writable(tokens, "tokens")
        a.tokens = tokens.data_ptr()
        a.token_stride = max(tokens.stride(0), a.max_draft + 1) if a.B <= 1 else tokens.stride(0)
        a.accepted = _dptr(accepted, torch.int32, a.B, "accepted", dev)
        a.row_status = _dptr(row_status, torch.int32, a.B, "row_status", dev)
        a.keep = (target_probs, draft_probs, draft_tokens, cu_draft, u_accept, u_sample, tokens, accepted, row_status)
        return a

    def apply(self, args: VerifyArgs, stream: Optional[torch.cuda.Stream] = None):
        """Enqueue one call on ``stream`` (default: current)."""
        _current(self.device)
        _check(self._L.clsample_verify(ctypes.byref(args), _stream_ptr(stream)))

    def __call__(self, target_probs, draft_tokens, cu_draft, u_accept, u_sample, *, max_draft: int,
                 draft_probs=None, stream=None) -> Dict[str, torch.Tensor]:
        """Verify, and return ``tokens`` int32 [B, max_draft + 1] (accepted tokens, the drawn
        token, then -1), ``accepted`` and ``status`` (int32 per request)."""
        B, dev = u_sample.numel(), target_probs.device
        with _on_stream(stream):
            out = {"tokens": torch.empty(B, int(max_draft) + 1, dtype=torch.int32, device=dev),
                   "accepted": torch.empty(B, dtype=torch.int32, device=dev),
                   "status": torch.empty(B, dtype=torch.int32, device=dev)}
        self.apply(self.make_args(target_probs, draft_tokens, cu_draft, u_accept, u_sample, max_draft=max_draft,
                                  draft_probs=draft_probs, tokens=out["tokens"], accepted=out["accepted"],
                                  row_status=out["status"]), stream)
        return out
