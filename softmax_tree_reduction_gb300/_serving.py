"""ctypes binding of the calls around the decode step (include/tree_attn.h):
norms and rotation of queries and keys, cache writes and reads, and attention
to selected pages.

As in ``_binding``, only argument marshalling: tensors are checked and turned
into pointers, missing outputs are allocated with torch, and the call is
enqueued on torch's current CUDA stream (or ``stream``).  The checks and the
descriptors of a layout are kept per thread and reused while the same shapes,
strides and types come back, so a serving loop pays for them once.
"""
from __future__ import annotations

import contextlib
import ctypes
import threading
from typing import Optional

import torch

from ._binding import (TA_F32, TaHeads, TaPagedKV, TaRope, TaShape, TaTokens, TreeAttnError, _dtype_code, load)

_PLANS_MAX = 256


class _Local(threading.local):
    def __init__(self):
        self.plans = {}


_local = _Local()


def _plan(key, make, *args):
    """This thread's plan for ``key`` (its structs are filled in and passed within one call)."""
    plans = _local.plans
    p = plans.get(key)
    if p is None:
        p = make(*args)
        if len(plans) >= _PLANS_MAX:
            plans.clear()
        plans[key] = p
    return p


def _device(*ts) -> int:
    """The CUDA device all of the tensors are on, which has to be the current one."""
    dev = ts[0].get_device()
    for t in ts:
        if t is not None and (t.get_device() != dev or dev < 0):
            raise ValueError("tensors must live on one CUDA device")
    if dev != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{dev}, which is not the current device: make it current first")
    return dev


def _on(stream, dev):
    """(stream handle, context in which tensors made belong to that stream)."""
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream, contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    if stream.device.index != dev:
        raise ValueError("the stream belongs to another device than the tensors")
    return stream.cuda_stream, torch.cuda.stream(stream)


def _vec_strides(t, what, output=False):
    """(token, head) strides of head vectors [T, H, d]."""
    if t.dim() != 3 or (t.stride(2) != 1 and t.numel()):
        raise ValueError(f"{what} must be [tokens, heads, head_dim] with contiguous channels")
    st, sh = (t.stride(i) if t.shape[i] > 1 else 0 for i in (0, 1))
    if output and ((t.shape[0] > 1 and st == 0) or (t.shape[1] > 1 and sh == 0)):
        raise ValueError(f"{what} is written to: its vectors must not share memory")
    return st, sh


def _ints(t, what, n):
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.shape[0] != n:
        raise ValueError(f"{what} must be a contiguous int32 tensor of {n} entries")


def _rope_struct(d, freq_n, inv_freq, q_weight, k_weight, norm, eps, interleaved) -> TaRope:
    if inv_freq is not None and (inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous()):
        raise ValueError("inv_freq must be a contiguous float32 tensor [rot_dim / 2]")
    wdt = None
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is None:
            continue
        if not norm:
            raise ValueError(f"{name} needs norm=True")
        if w.dtype not in (torch.bfloat16, torch.float32) or w.shape != (d,) or not w.is_contiguous() or (wdt or w.dtype) != w.dtype:
            raise ValueError("norm weights must be contiguous [head_dim] tensors of one type, bfloat16 or float32")
        wdt = w.dtype
    return TaRope(None, None, None, _dtype_code(wdt or torch.float32), 2 * freq_n, int(bool(interleaved)), int(bool(norm)), float(eps), 0)


def _set_rope(r, inv_freq, q_weight, k_weight):
    r.inv_freq = inv_freq.data_ptr() if inv_freq is not None else None
    r.q_weight = q_weight.data_ptr() if q_weight is not None else None
    r.k_weight = k_weight.data_ptr() if k_weight is not None else None


def _lay(t):
    """What of a tensor a plan depends on."""
    return None if t is None else (t.shape, t.stride(), t.dtype)


def _vec_dtype(t):
    if t.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"head vectors must be bfloat16 or float32, not {t.dtype}")
    return _dtype_code(t.dtype)


class _NormRopePlan:
    def __init__(self, q, k, q_out, k_out, positions, inv_freq, q_weight, k_weight, norm, eps, interleaved):
        if not norm and inv_freq is None:
            raise ValueError("nothing to do: no norm and no inv_freq")
        x = q if q is not None else k
        T, d = x.shape[0], x.shape[2] if x.dim() == 3 else 0
        _ints(positions, "positions", T)
        self.heads = []
        for name, a, o in (("q", q, q_out), ("k", k, k_out)):
            if a is None:
                if o is not None:
                    raise ValueError(f"{name}_out without {name}")
                self.heads += [None, None]
                continue
            if o.shape != a.shape or a.shape[0] != T or a.shape[2] != d or a.dtype != x.dtype or o.dtype != x.dtype:
                raise ValueError("q, k and their outputs must agree on tokens, head_dim and type")
            self.heads += [TaHeads(None, *_vec_strides(a, name)), TaHeads(None, *_vec_strides(o, name + "_out", True))]
        self.shape = TaShape(1, q.shape[1] if q is not None else 0, k.shape[1] if k is not None else 0, d, 1, _vec_dtype(x), TA_F32, 0.0, 0, 0, 0)
        self.tokens = TaTokens(T, 0, None, None)
        self.rope = _rope_struct(d, inv_freq.numel() if inv_freq is not None else 0, inv_freq, q_weight, k_weight, norm, eps, interleaved)
        self.args = [ctypes.byref(self.shape), ctypes.byref(self.tokens), ctypes.byref(self.rope),
                     *(ctypes.byref(h) if h is not None else None for h in self.heads)]


def tree_attn_norm_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor,
                        inv_freq: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                        k_weight: Optional[torch.Tensor] = None, norm: bool = True, eps: float = 1e-6,
                        interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                        k_out: Optional[torch.Tensor] = None, stream=None):
    """Per-head RMS norm and position rotation of queries and keys in one kernel.

    q: [T, Hq, d], k: [T, Hkv, d] (either may be None), BF16 or FP32, channels
    contiguous (views of a packed projection are fine); positions: int32 [T], negative
    for padding tokens, whose outputs are left as they were; inv_freq: float32
    [rot_dim / 2] (rot_dim a multiple of 16; None: no rotation); weights: [d] or None.
    Outputs may be the inputs themselves.  Returns (q_out, k_out); an output that is
    not passed is allocated (padding tokens then hold zeros).
    """
    lib = load()
    if q is None and k is None:
        raise ValueError("q or k is needed")
    dev = _device(positions, q, k, q_out, k_out, inv_freq, q_weight, k_weight)
    handle, ctx = _on(stream, dev)
    with ctx:
        if q is not None and q_out is None:
            q_out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        if k is not None and k_out is None:
            k_out = torch.zeros(k.shape, dtype=k.dtype, device=k.device)
    key = ("norm_rope", _lay(q), _lay(k), _lay(q_out), _lay(k_out), _lay(positions), _lay(inv_freq), _lay(q_weight), _lay(k_weight),
           norm, eps, interleaved)
    p = _plan(key, _NormRopePlan, q, k, q_out, k_out, positions, inv_freq, q_weight, k_weight, norm, eps, interleaved)
    p.tokens.positions = positions.data_ptr()
    _set_rope(p.rope, inv_freq, q_weight, k_weight)
    for h, t in zip(p.heads, (q, q_out, k, k_out)):
        if h is not None:
            h.data = t.data_ptr()
    rc = lib.tree_attn_norm_rope(*p.args, handle)
    if rc:
        raise TreeAttnError(rc, "tree_attn_norm_rope")
    return q_out, k_out


class _CachePlan:
    """Shape, pages and token list of a cache write or read."""

    def __init__(self, k_cache, v_cache, positions, rows, block_table, max_seqlen, vec, hq, k_scale, v_scale):
        if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or v_cache.stride() != k_cache.stride() or v_cache.dtype != k_cache.dtype:
            raise ValueError("k_cache and v_cache must be 4-D with the same shape, strides and type")
        if k_cache.stride(3) != 1:
            raise ValueError("cache channels must be contiguous")
        d = k_cache.shape[3]
        self.paged = None
        if block_table is None:
            B, hkv, S = k_cache.shape[:3]
            order = (0, 1, 2)                        # [B, Hkv, S, d]
        else:
            if block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous():
                raise ValueError("block_table must be a contiguous int32 [B, max_pages] tensor")
            pages, page, hkv = k_cache.shape[:3]     # [pages, page, Hkv, d]
            order = (0, 2, 1)
            B = block_table.shape[0]
            S = int(max_seqlen) if max_seqlen is not None else block_table.shape[1] * page
            self.paged = TaPagedKV(None, block_table.shape[1], page, pages, 0)
        sb, sh, st = (k_cache.stride(i) if k_cache.shape[i] > 1 else max(d, 16) for i in order)
        T = positions.shape[0] if positions.dim() == 1 else -1
        _ints(positions, "positions", T)
        if rows is not None:
            _ints(rows, "rows", T)
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is not None and (s.dtype != torch.float32 or s.shape != (hkv,) or not s.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous float32 tensor [num_kv_heads]")
        if vec.dim() != 3 or vec.shape != (T, hkv, d):
            raise ValueError("head vectors must be [tokens, num_kv_heads, head_dim] of the cache")
        self.shape = TaShape(B, hq if hq else hkv, hkv, d, S, _vec_dtype(vec), _dtype_code(k_cache.dtype), 0.0, sb, sh, st)
        self.tokens = TaTokens(T, 0, None, None)

    def base(self):
        return [ctypes.byref(self.shape), ctypes.byref(self.paged) if self.paged is not None else None, ctypes.byref(self.tokens)]

    def set(self, positions, rows, block_table):
        self.tokens.positions = positions.data_ptr()
        self.tokens.rows = rows.data_ptr() if rows is not None else None
        if self.paged is not None:
            self.paged.block_table = block_table.data_ptr()


class _WritePlan(_CachePlan):
    def __init__(self, k, v, k_cache, v_cache, positions, rows, block_table, max_seqlen, k_scale, v_scale, q, q_out, rope):
        if v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v must agree on shape and type")
        if q is not None and (rope is None or q.dim() != 3 or q.shape[0] != k.shape[0] or q.shape[2] != k.shape[2] or q.dtype != k.dtype
                              or q_out.shape != q.shape or q_out.dtype != q.dtype):
            raise ValueError("q needs a norm or rotation, and must agree with k and q_out on tokens, head_dim and type")
        super().__init__(k_cache, v_cache, positions, rows, block_table, max_seqlen, k, q.shape[1] if q is not None else 0, k_scale, v_scale)
        self.rope = None
        if rope is not None:
            inv_freq = rope[0]
            self.rope = _rope_struct(k.shape[2], inv_freq.numel() if inv_freq is not None else 0, *rope)
        self.heads = [None, None] if q is None else [TaHeads(None, *_vec_strides(q, "q")), TaHeads(None, *_vec_strides(q_out, "q_out", True))]
        self.heads += [TaHeads(None, *_vec_strides(k, "k")), TaHeads(None, *_vec_strides(v, "v"))]
        self.args = [*self.base(), ctypes.byref(self.rope) if self.rope is not None else None,
                     *(ctypes.byref(h) if h is not None else None for h in self.heads)]


def tree_attn_cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          positions: torch.Tensor, rows: Optional[torch.Tensor] = None,
                          block_table: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                          v_scale: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                          q_out: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
                          q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                          norm: bool = False, eps: float = 1e-6, interleaved: bool = False,
                          max_seqlen: Optional[int] = None, stream=None):
    """Store the keys and values of a token list in a dense or paged cache.

    k, v: [T, Hkv, d], BF16 or FP32; k_cache, v_cache: dense [B, Hkv, S, d] views, or page
    pools [num_pages, page_size, Hkv, d] with ``block_table``, of any cache type (E4M3 with
    ``k_scale``/``v_scale``: codes are e4m3(x / scale), saturating); positions: int32 [T]
    (negative: padding, nothing is stored); rows: int32 [T] batch rows (None: token t
    is row t's).  With ``inv_freq`` or ``norm`` the keys are rotated or normed first, and so
    are the queries ``q`` [T, Hq, d] when given (into ``q_out``, which may be q), all in one
    kernel.  Returns q_out (None without q).
    """
    lib = load()
    rope = (inv_freq, q_weight, k_weight, norm, eps, interleaved) if norm or inv_freq is not None else None
    if rope is None and (q_weight is not None or k_weight is not None):
        raise ValueError("norm weights need norm=True")
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    dev = _device(k, v, k_cache, v_cache, positions, rows, block_table, k_scale, v_scale, q, q_out, inv_freq, q_weight, k_weight)
    handle, ctx = _on(stream, dev)
    if q is not None and q_out is None:
        with ctx:
            q_out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    key = ("write", _lay(k), _lay(v), _lay(k_cache), _lay(v_cache), _lay(positions), _lay(rows), _lay(block_table), _lay(k_scale),
           _lay(v_scale), _lay(q), _lay(q_out), _lay(inv_freq), _lay(q_weight), _lay(k_weight), norm, eps, interleaved, max_seqlen)
    p = _plan(key, _WritePlan, k, v, k_cache, v_cache, positions, rows, block_table, max_seqlen, k_scale, v_scale, q, q_out, rope)
    p.set(positions, rows, block_table)
    if p.rope is not None:
        _set_rope(p.rope, inv_freq, q_weight, k_weight)
    for h, t in zip(p.heads, (q, q_out, k, v)):
        if h is not None:
            h.data = t.data_ptr()
    rc = lib.tree_attn_cache_write(*p.args, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr() if k_scale is not None else None,
                                   v_scale.data_ptr() if v_scale is not None else None, handle)
    if rc:
        raise TreeAttnError(rc, "tree_attn_cache_write")
    return q_out


class _ReadPlan(_CachePlan):
    def __init__(self, k_cache, v_cache, positions, rows, block_table, max_seqlen, k_scale, v_scale, k_out, v_out):
        if v_out.shape != k_out.shape or v_out.dtype != k_out.dtype:
            raise ValueError("k_out and v_out must agree on shape and type")
        super().__init__(k_cache, v_cache, positions, rows, block_table, max_seqlen, k_out, 0, k_scale, v_scale)
        self.outs = [TaHeads(None, *_vec_strides(k_out, "k_out", True)), TaHeads(None, *_vec_strides(v_out, "v_out", True))]
        self.args = self.base()
        self.out_args = [ctypes.byref(h) for h in self.outs]


def tree_attn_cache_read(k_cache: torch.Tensor, v_cache: torch.Tensor, positions: torch.Tensor,
                         rows: Optional[torch.Tensor] = None, block_table: Optional[torch.Tensor] = None,
                         k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                         dtype: torch.dtype = torch.bfloat16, k_out: Optional[torch.Tensor] = None,
                         v_out: Optional[torch.Tensor] = None, max_seqlen: Optional[int] = None, stream=None):
    """Read the keys and values of a token list from a dense or paged cache.

    The caches, positions, rows and block_table are those of tree_attn_cache_write.
    Returns (k_out, v_out), [T, Hkv, d] of ``dtype`` (BF16 or FP32) unless passed; E4M3 codes
    are multiplied by their head's scale.  Vectors of padding tokens are left as they were
    (zeros in outputs allocated here).
    """
    lib = load()
    dev = _device(k_cache, v_cache, positions, rows, block_table, k_scale, v_scale, k_out, v_out)
    handle, ctx = _on(stream, dev)
    if k_out is None or v_out is None:
        size = (positions.shape[0], k_cache.shape[1] if block_table is None else k_cache.shape[2], k_cache.shape[3])
        with ctx:
            like = k_out if k_out is not None else v_out
            dt = dtype if like is None else like.dtype
            k_out = torch.zeros(size, dtype=dt, device=k_cache.device) if k_out is None else k_out
            v_out = torch.zeros(size, dtype=dt, device=k_cache.device) if v_out is None else v_out
    key = ("read", _lay(k_cache), _lay(v_cache), _lay(positions), _lay(rows), _lay(block_table), _lay(k_scale), _lay(v_scale),
           _lay(k_out), _lay(v_out), max_seqlen)
    p = _plan(key, _ReadPlan, k_cache, v_cache, positions, rows, block_table, max_seqlen, k_scale, v_scale, k_out, v_out)
    p.set(positions, rows, block_table)
    p.outs[0].data, p.outs[1].data = k_out.data_ptr(), v_out.data_ptr()
    rc = lib.tree_attn_cache_read(*p.args, k_cache.data_ptr(), v_cache.data_ptr(), *p.out_args,
                                  k_scale.data_ptr() if k_scale is not None else None,
                                  v_scale.data_ptr() if v_scale is not None else None, handle)
    if rc:
        raise TreeAttnError(rc, "tree_attn_cache_read")
    return k_out, v_out


class _PagesPlan:
    """Shape and pages of a call on a paged cache's selected pages."""

    def __init__(self, q, hkv, d, kv_code, strides, page, pages, block_table, seqlens, max_seqlen, scale):
        if block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous():
            raise ValueError("block_table must be a contiguous int32 [B, max_pages] tensor")
        B = block_table.shape[0]
        _ints(seqlens, "seqlens", B)
        hq, qcode = hkv, TA_F32
        if q is not None:
            if q.dim() != 3 or not q.is_contiguous() or q.shape[0] != B or q.shape[2] != d:
                raise ValueError("q must be a contiguous [B, Hq, d] tensor that agrees with the pages and block_table")
            hq, qcode = q.shape[1], _vec_dtype(q)
        S = int(max_seqlen) if max_seqlen is not None else block_table.shape[1] * page
        self.shape = TaShape(B, hq, hkv, d, S, qcode, kv_code, float(scale or 0.0), *strides)
        self.paged = TaPagedKV(None, block_table.shape[1], page, pages, 0)
        self.args = (ctypes.byref(self.shape), ctypes.byref(self.paged))


def _pool(k_pages):
    """(page stride, head stride, token stride) of a [num_pages, page_size, Hkv, d] pool."""
    if k_pages.dim() != 4 or k_pages.stride(3) != 1:
        raise ValueError("page pools must be [num_pages, page_size, Hkv, d] with contiguous channels")
    return tuple(k_pages.stride(i) if k_pages.shape[i] > 1 else max(k_pages.shape[3], 16) for i in (0, 2, 1))


class _BoundsPlan(_PagesPlan):
    def __init__(self, k_pages, block_table, seqlens, bounds, max_seqlen):
        pages, page, hkv, d = k_pages.shape
        code = _dtype_code(k_pages.dtype)
        want = torch.float32 if code == TA_F32 else torch.bfloat16
        if bounds.shape != (pages, hkv, 2, d) or bounds.dtype != want or not bounds.is_contiguous():
            raise ValueError(f"bounds must be a contiguous {want} [num_pages, Hkv, 2, d] tensor")
        super().__init__(None, hkv, d, code, _pool(k_pages), page, pages, block_table, seqlens, max_seqlen, None)


def tree_attn_page_bounds(k_pages: torch.Tensor, block_table: torch.Tensor, seqlens: torch.Tensor,
                          bounds: Optional[torch.Tensor] = None, new_tokens: int = 0,
                          max_seqlen: Optional[int] = None, stream=None):
    """Channel minima and maxima of the keys of each row's pages, [num_pages, Hkv, 2, d].

    k_pages: [num_pages, page_size, Hkv, d]; only the pages holding a row's last ``new_tokens``
    tokens are updated (<= 0: all of its pages), each over all of its valid tokens.  bounds is
    FP32 for FP32 caches, else BF16 (codes of E4M3 caches, without the scale); allocated as
    zeros when not passed.  Returns bounds.
    """
    lib = load()
    dev = _device(k_pages, block_table, seqlens, bounds)
    handle, ctx = _on(stream, dev)
    if bounds is None:
        if k_pages.dim() != 4:
            raise ValueError("page pools must be [num_pages, page_size, Hkv, d]")
        with ctx:
            bounds = torch.zeros((k_pages.shape[0], k_pages.shape[2], 2, k_pages.shape[3]), device=k_pages.device,
                                 dtype=torch.float32 if k_pages.dtype == torch.float32 else torch.bfloat16)
    _pool(k_pages)
    p = _plan(("bounds", _lay(k_pages), _lay(block_table), _lay(seqlens), _lay(bounds), max_seqlen), _BoundsPlan, k_pages, block_table,
              seqlens, bounds, max_seqlen)
    p.paged.block_table = block_table.data_ptr()
    rc = lib.tree_attn_page_bounds(*p.args, k_pages.data_ptr(), seqlens.data_ptr(), max(0, int(new_tokens)), bounds.data_ptr(), handle)
    if rc:
        raise TreeAttnError(rc, "tree_attn_page_bounds")
    return bounds


class _SelectPlan(_PagesPlan):
    def __init__(self, q, bounds, block_table, seqlens, page, num_select, max_seqlen, selected):
        if bounds.dim() != 4 or bounds.shape[2] != 2 or not bounds.is_contiguous() or bounds.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("bounds must be a contiguous float32 or bfloat16 [num_pages, Hkv, 2, d] tensor")
        pages, hkv, _, d = bounds.shape
        if selected.shape != (block_table.shape[0], hkv, num_select) or selected.dtype != torch.int32 or not selected.is_contiguous():
            raise ValueError("selected must be a contiguous int32 [B, Hkv, num_select] tensor")
        super().__init__(q, hkv, d, _dtype_code(bounds.dtype), (0, 0, 0), page, pages, block_table, seqlens, max_seqlen, None)
        self.ws_bytes = int(load().tree_attn_select_workspace_bytes(*self._with_table(block_table)))

    def _with_table(self, block_table):
        self.paged.block_table = block_table.data_ptr()
        return self.args


def tree_attn_select_pages(q: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, seqlens: torch.Tensor,
                           page_size: int, num_select: int, first_pages: int = 1, last_pages: int = 1,
                           selected: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                           max_seqlen: Optional[int] = None, stream=None):
    """The logical pages each (row, KV head) should attend to, int32 [B, Hkv, num_select].

    q: [B, Hq, d]; bounds as kept by tree_attn_page_bounds.  The first and last pages are always
    listed; the others by the sum over the head group of an upper bound of the page's logits.
    Ascending, -1 behind the listed pages.  ``workspace``: a CUDA tensor of at least
    tree_attn_select_workspace_bytes bytes (allocated when not passed).
    """
    lib = load()
    dev = _device(q, bounds, block_table, seqlens, selected, workspace)
    handle, ctx = _on(stream, dev)
    page_size, num_select = int(page_size), int(num_select)
    if selected is None:
        with ctx:
            selected = torch.empty((block_table.shape[0], bounds.shape[1], max(0, num_select)), dtype=torch.int32, device=q.device)
    p = _plan(("select", _lay(q), _lay(bounds), _lay(block_table), _lay(seqlens), page_size, num_select, max_seqlen, _lay(selected)),
              _SelectPlan, q, bounds, block_table, seqlens, page_size, num_select, max_seqlen, selected)
    p.paged.block_table = block_table.data_ptr()
    if workspace is None:
        with ctx:
            workspace = torch.empty(max(16, p.ws_bytes), dtype=torch.uint8, device=q.device)
    rc = lib.tree_attn_select_pages(*p.args, q.data_ptr(), bounds.data_ptr(), seqlens.data_ptr(), num_select, int(first_pages),
                                    int(last_pages), selected.data_ptr(), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), handle)
    if rc:
        raise TreeAttnError(rc, "tree_attn_select_pages")
    return selected


def tree_attn_select_workspace_bytes(batch: int, num_kv_heads: int, max_pages: int) -> int:
    """Bytes tree_attn_select_pages needs as workspace for rows of up to ``max_pages`` pages."""
    shape = TaShape(batch, num_kv_heads, num_kv_heads, 128, max_pages * 16, TA_F32, TA_F32, 0.0, 0, 0, 0)
    paged = TaPagedKV(16, max_pages, 16, 1, 0)   # (a table address is required, none is read)
    return int(load().tree_attn_select_workspace_bytes(ctypes.byref(shape), ctypes.byref(paged)))


class _DecodePlan(_PagesPlan):
    def __init__(self, q, k_pages, v_pages, block_table, seqlens, selected, max_seqlen, scale, k_scale, v_scale, out, lse):
        if v_pages.shape != k_pages.shape or v_pages.stride() != k_pages.stride() or v_pages.dtype != k_pages.dtype:
            raise ValueError("k_pages and v_pages must agree on shape, strides and type")
        strides = _pool(k_pages)
        pages, page, hkv, d = k_pages.shape
        B = block_table.shape[0]
        if selected.dim() != 3 or selected.shape[:2] != (B, hkv) or selected.dtype != torch.int32 or not selected.is_contiguous():
            raise ValueError("selected must be a contiguous int32 [B, Hkv, num_select] tensor")
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is not None and (s.dtype != torch.float32 or s.shape != (hkv,) or not s.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous float32 tensor [num_kv_heads]")
        super().__init__(q, hkv, d, _dtype_code(k_pages.dtype), strides, page, pages, block_table, seqlens, max_seqlen, scale)
        hq = q.shape[1]
        if out.shape != (B, hq, d) or out.dtype != torch.float32 or not out.is_contiguous():
            raise ValueError("out must be a contiguous float32 [B, Hq, d] tensor")
        if lse is not None and (lse.shape != (B, hq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
            raise ValueError("lse must be a contiguous float32 [B, Hq] tensor")


def tree_attn_decode_selected(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                              seqlens: torch.Tensor, selected: torch.Tensor, out: Optional[torch.Tensor] = None,
                              lse: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                              max_seqlen: Optional[int] = None, k_scale: Optional[torch.Tensor] = None,
                              v_scale: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """Decode attention over the listed pages; returns (out [B, Hq, d] fp32, lse [B, Hq] fp32 or None).

    selected: int32 [B, Hkv, num_select] logical pages per row and KV head (negative entries and
    pages past the row's end hold no token); the other arguments are tree_attn_decode_paged's.
    """
    lib = load()
    dev = _device(q, k_pages, v_pages, block_table, seqlens, selected, out, lse, k_scale, v_scale)
    handle, ctx = _on(stream, dev)
    if out is None or (lse is None and want_lse):
        with ctx:
            if out is None:
                out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
            if lse is None and want_lse:
                lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    key = ("decode", _lay(q), _lay(k_pages), _lay(v_pages), _lay(block_table), _lay(seqlens), _lay(selected), max_seqlen, scale,
           _lay(k_scale), _lay(v_scale), _lay(out), _lay(lse))
    p = _plan(key, _DecodePlan, q, k_pages, v_pages, block_table, seqlens, selected, max_seqlen, scale, k_scale, v_scale, out, lse)
    p.paged.block_table = block_table.data_ptr()
    rc = lib.tree_attn_decode_selected(*p.args, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), seqlens.data_ptr(),
                                       selected.data_ptr(), selected.shape[2], out.data_ptr(), lse.data_ptr() if lse is not None else None,
                                       k_scale.data_ptr() if k_scale is not None else None,
                                       v_scale.data_ptr() if v_scale is not None else None, handle)
    if rc:
        raise TreeAttnError(rc, "tree_attn_decode_selected")
    return out, lse
