"""Binding of the calls around the decode step (include/tree_attn.h): norms and
rotation of queries and keys, cache writes and reads, and attention to
selected pages.

As in ``_binding``, only argument marshalling: missing outputs are allocated
with torch, and the call is enqueued on torch's current CUDA stream (or
``stream``).  The checks and descriptors are made by the extension module
``_serving_calls`` (csrc/serving_calls.cpp), which costs well under a
microsecond; through ctypes they took longer than the kernels.  Arguments that
the descriptors cannot express raise ValueError or TypeError, the library's own
refusals TreeAttnError.
"""
from __future__ import annotations

import contextlib
import ctypes
import threading
from typing import Optional

import torch

from ._binding import LIB_PATH, TA_F32, TaPagedKV, TaShape, TreeAttnError, load

_calls = None
_lock = threading.Lock()


def _open():
    """The extension module, bound to the loaded library."""
    global _calls
    with _lock:
        if _calls is None:
            load()
            try:
                from . import _serving_calls as mod
            except ImportError as e:
                raise RuntimeError("the extension module _serving_calls is missing: build it with "
                                   "`python -m softmax_tree_reduction_gb300.build`") from e
            mod.init(LIB_PATH)
            _calls = mod
    return _calls


def _on(stream, like: torch.Tensor):
    """(stream handle or None, context in which tensors made belong to that stream)."""
    if stream is None:
        return None, contextlib.nullcontext()
    if not like.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    if stream.device != like.device:
        raise ValueError("the stream belongs to another device than the tensors")
    return stream.cuda_stream, torch.cuda.stream(stream)


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
    if stream is not None or (q is not None and q_out is None) or (k is not None and k_out is None):
        stream, ctx = _on(stream, positions)
        with ctx:
            if q is not None and q_out is None:
                q_out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
            if k is not None and k_out is None:
                k_out = torch.zeros(k.shape, dtype=k.dtype, device=k.device)
    rc = (_calls or _open()).norm_rope(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, interleaved, q_out, k_out, stream)
    if rc:
        raise TreeAttnError(rc, "tree_attn_norm_rope")
    return q_out, k_out


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
    is row t's); max_seqlen: positions from it on are out of range (default: all that the cache
    or the block table holds).  With ``inv_freq`` or ``norm`` the keys are rotated or normed first, and so
    are the queries ``q`` [T, Hq, d] when given (into ``q_out``, which may be q), all in one
    kernel.  Returns q_out (None without q).
    """
    if stream is not None or (q is not None and q_out is None):
        stream, ctx = _on(stream, k)
        if q is not None and q_out is None:
            with ctx:
                q_out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    rc = (_calls or _open()).cache_write(k, v, k_cache, v_cache, positions, rows, block_table, k_scale, v_scale, q, q_out, inv_freq, q_weight,
                                         k_weight, norm, eps, interleaved, max_seqlen, stream)
    if rc:
        raise TreeAttnError(rc, "tree_attn_cache_write")
    return q_out


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
    if stream is not None or k_out is None or v_out is None:
        if k_cache.dim() != 4:
            raise ValueError("caches must be 4-D")
        stream, ctx = _on(stream, k_cache)
        like = k_out if k_out is not None else v_out
        size = (positions.shape[0], k_cache.shape[1] if block_table is None else k_cache.shape[2], k_cache.shape[3])
        with ctx:
            dt = dtype if like is None else like.dtype
            k_out = torch.zeros(size, dtype=dt, device=k_cache.device) if k_out is None else k_out
            v_out = torch.zeros(size, dtype=dt, device=k_cache.device) if v_out is None else v_out
    rc = (_calls or _open()).cache_read(k_cache, v_cache, positions, rows, block_table, k_scale, v_scale, k_out, v_out, max_seqlen, stream)
    if rc:
        raise TreeAttnError(rc, "tree_attn_cache_read")
    return k_out, v_out


def tree_attn_page_bounds(k_pages: torch.Tensor, block_table: torch.Tensor, seqlens: torch.Tensor,
                          bounds: Optional[torch.Tensor] = None, new_tokens: int = 0,
                          max_seqlen: Optional[int] = None, stream=None):
    """Channel minima and maxima of the keys of each row's pages, [num_pages, Hkv, 2, d].

    k_pages: [num_pages, page_size, Hkv, d]; only the pages holding a row's last ``new_tokens``
    tokens are updated (<= 0: all of its pages), each over all of its valid tokens.  bounds is
    FP32 for FP32 caches, else BF16 (codes of E4M3 caches, without the scale); allocated as
    zeros when not passed.  Returns bounds.
    """
    if stream is not None or bounds is None:
        if k_pages.dim() != 4:
            raise ValueError("page pools must be [num_pages, page_size, Hkv, d]")
        stream, ctx = _on(stream, k_pages)
        if bounds is None:
            with ctx:
                bounds = torch.zeros((k_pages.shape[0], k_pages.shape[2], 2, k_pages.shape[3]), device=k_pages.device,
                                     dtype=torch.float32 if k_pages.dtype == torch.float32 else torch.bfloat16)
    rc = (_calls or _open()).page_bounds(k_pages, block_table, seqlens, bounds, new_tokens, max_seqlen, stream)
    if rc:
        raise TreeAttnError(rc, "tree_attn_page_bounds")
    return bounds


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
    calls = _calls or _open()
    if stream is not None or selected is None:
        stream, ctx = _on(stream, q)
        with ctx:
            if selected is None:
                selected = torch.empty((block_table.shape[0], bounds.shape[1], max(0, int(num_select))), dtype=torch.int32, device=q.device)
            if workspace is None and stream is not None:   # (on the current stream the extension allocates it)
                workspace = torch.empty(max(16, calls.select_workspace_bytes(bounds, block_table, page_size, max_seqlen)), dtype=torch.uint8,
                                        device=q.device)
    rc = calls.select_pages(q, bounds, block_table, seqlens, page_size, num_select, first_pages, last_pages, selected, workspace, max_seqlen, stream)
    if rc:
        raise TreeAttnError(rc, "tree_attn_select_pages")
    return selected


def tree_attn_select_workspace_bytes(batch: int, num_kv_heads: int, max_pages: int) -> int:
    """Bytes tree_attn_select_pages needs as workspace for rows of up to ``max_pages`` pages."""
    most = 2 ** 31 - 1                           # tokens of a row; more pages than they fill are not used
    if max(batch, num_kv_heads, max_pages) > most:
        raise ValueError("batch, num_kv_heads and max_pages must be below 2^31")
    if min(batch, num_kv_heads, max_pages) < 1:
        return 0
    shape = TaShape(batch, num_kv_heads, num_kv_heads, 128, min(max_pages * 16, most), TA_F32, TA_F32, 0.0, 0, 0, 0)
    paged = TaPagedKV(16, max_pages, 16, 1, 0)   # (a table address is required, none is read)
    return int(load().tree_attn_select_workspace_bytes(ctypes.byref(shape), ctypes.byref(paged)))


def tree_attn_decode_selected(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                              seqlens: torch.Tensor, selected: torch.Tensor, out: Optional[torch.Tensor] = None,
                              lse: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                              max_seqlen: Optional[int] = None, k_scale: Optional[torch.Tensor] = None,
                              v_scale: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """Decode attention over the listed pages; returns (out [B, Hq, d] fp32, lse [B, Hq] fp32 or None).

    selected: int32 [B, Hkv, num_select] logical pages per row and KV head (negative entries and
    pages past the row's end hold no token); the other arguments are tree_attn_decode_paged's.
    """
    if stream is not None or out is None or (lse is None and want_lse):
        stream, ctx = _on(stream, q)
        with ctx:
            if out is None:
                out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
            if lse is None and want_lse:
                lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    rc = (_calls or _open()).decode_selected(q, k_pages, v_pages, block_table, seqlens, selected, out, lse, scale, max_seqlen, k_scale, v_scale, stream)
    if rc:
        raise TreeAttnError(rc, "tree_attn_decode_selected")
    return out, lse


def tree_attn_cache_write_int4(k: torch.Tensor, v: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor,
                               k_steps: torch.Tensor, v_steps: torch.Tensor, positions: torch.Tensor,
                               rows: Optional[torch.Tensor] = None, block_table: Optional[torch.Tensor] = None,
                               k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                               q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                               inv_freq: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                               k_weight: Optional[torch.Tensor] = None, norm: bool = False, eps: float = 1e-6,
                               interleaved: bool = False, max_seqlen: Optional[int] = None, stream=None):
    """Store the keys and values of a token list in a 4-bit cache.

    The cache is codes, uint8 [B, Hkv, S, d / 2] or pools [num_pages, page_size, Hkv, d / 2] with
    ``block_table`` (two channels a byte, the even one in the low half), and steps, float8_e4m3fn
    [.., d / 16]; a channel's value is scale * step * (code - 8) with the FP32 scale of its KV head
    (``k_scale``/``v_scale``, both or neither).  Each 16 channels get the step next to a seventh of
    their largest magnitude and the codes next to their quotients by it.  Steps lie between 2^-9 and 448 and
    are coarse below 2^-6: heads whose vectors are small (below about 0.05) want a scale, for instance their
    largest magnitude / 448.  The other arguments are tree_attn_cache_write's.  Returns q_out (None without q).
    """
    if stream is not None or (q is not None and q_out is None):
        stream, ctx = _on(stream, k)
        if q is not None and q_out is None:
            with ctx:
                q_out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    rc = (_calls or _open()).cache_write_int4(k, v, k_codes, v_codes, k_steps, v_steps, positions, rows, block_table, k_scale, v_scale, q, q_out,
                                              inv_freq, q_weight, k_weight, norm, eps, interleaved, max_seqlen, stream)
    if rc:
        raise TreeAttnError(rc, "tree_attn_cache_write_int4")
    return q_out


def tree_attn_cache_read_int4(k_codes: torch.Tensor, v_codes: torch.Tensor, k_steps: torch.Tensor, v_steps: torch.Tensor,
                              positions: torch.Tensor, rows: Optional[torch.Tensor] = None,
                              block_table: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                              v_scale: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                              k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                              max_seqlen: Optional[int] = None, stream=None):
    """Read the keys and values of a token list from a 4-bit cache (tree_attn_cache_write_int4).

    Returns (k_out, v_out), [T, Hkv, d] of ``dtype`` (BF16 or FP32) unless passed; vectors of padding
    tokens are left as they were (zeros in outputs allocated here).
    """
    if stream is not None or k_out is None or v_out is None:
        if k_codes.dim() != 4:
            raise ValueError("4-bit caches must be 4-D")
        stream, ctx = _on(stream, k_codes)
        like = k_out if k_out is not None else v_out
        size = (positions.shape[0], k_codes.shape[1] if block_table is None else k_codes.shape[2], 2 * k_codes.shape[3])
        with ctx:
            dt = dtype if like is None else like.dtype
            k_out = torch.zeros(size, dtype=dt, device=k_codes.device) if k_out is None else k_out
            v_out = torch.zeros(size, dtype=dt, device=k_codes.device) if v_out is None else v_out
    rc = (_calls or _open()).cache_read_int4(k_codes, v_codes, k_steps, v_steps, positions, rows, block_table, k_scale, v_scale, k_out, v_out,
                                             max_seqlen, stream)
    if rc:
        raise TreeAttnError(rc, "tree_attn_cache_read_int4")
    return k_out, v_out


def _windowed_buffers(q, cache, block_table, window, sinks, max_seqlen, out, lse, want_lse, workspace, stream):
    """Outputs that were not passed, and with an explicit stream the workspace too (else the extension makes it)."""
    if stream is not None or out is None or (lse is None and want_lse):
        calls = _calls or _open()
        stream, ctx = _on(stream, q)
        with ctx:
            if out is None:
                out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
            if lse is None and want_lse:
                lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
            if workspace is None and stream is not None:
                need = calls.window_workspace_bytes(cache, block_table, q, window, sinks, max_seqlen)
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    return out, lse, workspace, stream


def tree_attn_decode_window(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, seqlens: torch.Tensor,
                            window: int, sinks: int = 0, block_table: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            scale: Optional[float] = None, max_seqlen: Optional[int] = None,
                            k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """Decode attention to the last ``window`` tokens and the first ``sinks`` ones.

    q: [B, Hq, d], or [B, Hq, nq, d] for several queries a row; query i sits at position
    s = seqlens[b] - nq + i and sees the tokens t <= s with t > s - window or t < sinks.  Caches: dense
    [B, Hkv, S, d] or pools [num_pages, page_size, Hkv, d] with ``block_table``, whose entries are read
    only for pages that some query sees: those that fell out of the window may be freed.  BF16 q with a BF16 or
    E4M3 cache (``k_scale``, ``v_scale``), FP32 q with an FP32 one.  ``workspace``: a CUDA tensor of at
    least tree_attn_window_workspace_bytes bytes (allocated when not passed).
    Returns (out fp32 of q's shape, lse fp32 without the channels, or None).
    """
    out, lse, workspace, stream = _windowed_buffers(q, k_cache, block_table, window, sinks, max_seqlen, out, lse, want_lse, workspace, stream)
    rc = (_calls or _open()).decode_window(q, k_cache, v_cache, seqlens, window, sinks, block_table, out, lse, scale, max_seqlen, k_scale, v_scale,
                                           workspace, stream)
    if rc:
        raise TreeAttnError(rc, "tree_attn_decode_window")
    return out, lse


def tree_attn_decode_int4(q: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor, k_steps: torch.Tensor,
                          v_steps: torch.Tensor, seqlens: torch.Tensor, window: Optional[int] = None, sinks: int = 0,
                          block_table: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                          max_seqlen: Optional[int] = None, k_scale: Optional[torch.Tensor] = None,
                          v_scale: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          want_lse: bool = True, stream=None):
    """Decode attention over a 4-bit cache (tree_attn_cache_write_int4), to all of a row or a window of it.

    q (BF16), outputs, window and sinks are tree_attn_decode_window's; ``window`` None: every token
    up to the query's own position.
    """
    out, lse, workspace, stream = _windowed_buffers(q, k_codes, block_table, window, sinks, max_seqlen, out, lse, want_lse, workspace, stream)
    rc = (_calls or _open()).decode_int4(q, k_codes, v_codes, k_steps, v_steps, seqlens, window, sinks, block_table, out, lse, scale, max_seqlen,
                                         k_scale, v_scale, workspace, stream)
    if rc:
        raise TreeAttnError(rc, "tree_attn_decode_int4")
    return out, lse


def tree_attn_window_workspace_bytes(q: torch.Tensor, cache: torch.Tensor, window: Optional[int] = None, sinks: int = 0,
                                     block_table: Optional[torch.Tensor] = None, max_seqlen: Optional[int] = None) -> int:
    """Bytes of workspace that tree_attn_decode_window (``cache``: its keys) or tree_attn_decode_int4 (its key
    codes) needs for these queries on the current device; 0: none."""
    return int((_calls or _open()).window_workspace_bytes(cache, block_table, q, window, sinks, max_seqlen))
