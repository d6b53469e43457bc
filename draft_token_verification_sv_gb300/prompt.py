"""PyTorch-facing wrappers of rotary positions and of the attention of prompts
(argument marshalling only; see include/spec_verify.h).

Rows of tokens come as [B, n, heads, dim] tensors or, packed, as
[total, heads, dim], with any row and head strides.  As in kvcache.py a call's
checks depend on shapes, strides and types alone and are made once for each
combination.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native as N
from .kvcache import (_KEPT, _PER_SEQUENCE, _at, _call, _contiguous, _count, _empty, _int32, _meta, _new, _numel, _one_device,
                      _rows, _see, _stream_of)
from .verify import _code


def _empty_like(x, stream):
    """A contiguous result of x's shape and type (see _empty)."""
    return _empty(x.shape, x.dtype, x.device, stream)


def _token_rows(m, name):
    """_rows of [B, n, heads, dim] or [total, heads, dim], whichever it is."""
    if len(m.shape) not in (3, 4):
        raise ValueError(f"{name} must be [total, heads, dim] or [B, n, heads, dim]")
    return _rows(m, name, m.shape[0], len(m.shape) == 3)


@functools.lru_cache(maxsize=_KEPT)
def _rope_plan(q, k, positions, inv_freq, sections, axis, adjacent, q_out, k_out):
    """q_out None: the call makes its results itself."""
    q, k, p, f = _see(q, "q"), _see(k, "k"), _see(positions, "positions"), _see(inv_freq, "inv_freq")
    q_out, k_out = _see(q_out, "out[0]"), _see(k_out, "out[1]")
    lead = q.shape[:-2]
    rows, heads, dim, *q_strides = _token_rows(q, "q")
    if f.dtype != torch.float32 or len(f.shape) != 1 or not _contiguous(f) or not 1 <= f.shape[0] <= dim // 2:
        raise ValueError("inv_freq must be a contiguous float32 tensor of at most dim / 2 entries")
    half = f.shape[0]
    axes = 1 if len(p.shape) == len(lead) else p.shape[0] if len(p.shape) == len(lead) + 1 else 0
    if p.dtype != torch.int32 or not _contiguous(p) or tuple(p.shape) not in (tuple(lead), (axes, *lead)):
        raise ValueError("positions must be a contiguous int32 tensor with one entry for each token, or [axes, ...] of such")
    if not 1 <= axes <= N.SV_MAX_ROPE_AXES:
        raise ValueError(f"positions may have 1 to {N.SV_MAX_ROPE_AXES} axes")
    if axis is None:
        sections = (half,) if sections is None and axes == 1 else sections
        if sections is None or len(sections) != axes or min(sections) < 0 or sum(sections) != half:
            raise ValueError("sections must have one entry for each axis of positions, and inv_freq's length as their sum")
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    elif sections is not None or len(axis) != half or min(axis) < 0 or max(axis) >= axes:
        raise ValueError("axis must have one entry for each of inv_freq, which is an axis of positions, and takes the place of sections")
    q_out_strides, k_heads, k_strides, k_out_strides = (heads * dim, dim), 0, (dim, dim), (dim, dim)
    if q_out is not None:
        if q_out.shape != q.shape or q_out.dtype != q.dtype:
            raise ValueError("out[0] must match q in shape and dtype")
        _, _, _, *q_out_strides = _token_rows(q_out, "out[0]")
    if k is not None:
        k_rows, k_heads, k_dim, *k_strides = _token_rows(k, "k")
        if k.shape[:-2] != lead or k_dim != dim or k.dtype != q.dtype:
            raise ValueError("k must match q in tokens, dim and dtype")
        k_out_strides = (k_heads * dim, dim)
        if q_out is not None:
            if k_out is None or k_out.shape != k.shape or k_out.dtype != k.dtype:
                raise ValueError("out[1] must match k in shape and dtype")
            _, _, _, *k_out_strides = _token_rows(k_out, "out[1]")
    d = N.RopeDesc(rows, heads, k_heads, dim, 2 * half, axes, int(adjacent), _code(q), rows, *q_strides, *k_strides,
                   *q_out_strides, *k_out_strides)
    d.axis[:half] = axis
    return ctypes.byref(d), _one_device(q, k, p, f, q_out, k_out)


def rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor, *,
         sections: tuple | None = None, axis: tuple | None = None, adjacent: bool = False, out: tuple | None = None, stream=None):
    """Rotary position embedding of queries and keys; see sv_rope.

    q [..., heads, dim], k [..., kv_heads, dim] or None, float32 or bfloat16;
    ``positions`` int32 [...], or [axes, ...] with ``sections``: how many pairs,
    one after the other, turn with each axis, or with ``axis``: the axis of each
    pair.  ``inv_freq`` float32 holds the radians a position of every pair; dims
    beyond 2 * len(inv_freq) stay.
    Pairs are (i, i + len(inv_freq)), with ``adjacent`` (2i, 2i + 1).  Returns
    (q, k) in new memory, or in ``out``, which may be (q, k) themselves."""
    q_out, k_out = (None, None) if out is None else out
    if out is not None and q_out is None:
        raise ValueError("out must be (q's result, k's)")
    d, gpu = _rope_plan(_meta(q), _meta(k), _meta(positions), _meta(inv_freq),
                        None if sections is None else tuple(int(n) for n in sections), None if axis is None else tuple(int(a) for a in axis),
                        bool(adjacent), _meta(q_out), _meta(k_out))
    if out is None:
        q_out, k_out = _empty_like(q, stream), None if k is None else _empty_like(k, stream)
    _call(gpu, "sv_rope", d, q.data_ptr(), _at(k), positions.data_ptr(), inv_freq.data_ptr(), q_out.data_ptr(),
          None if k is None else k_out.data_ptr(), _stream_of(stream, gpu))
    return q_out, None if k is None else k_out


@functools.lru_cache(maxsize=_KEPT)
def _prompt_plan(q, k, v, start, max_new, scale, window, sinks, out, status):
    """out None: the call makes its result itself."""
    q, k, v, out = _see(q, "q"), _see(k, "k"), _see(v, "v"), _see(out, "out")
    ragged = start is not None
    if not ragged and len(q.shape) != 4:
        raise ValueError("q must be [B, n, heads, dim], or [total, heads, dim] with new_start")
    B = _numel(_see(start, "new_start").shape) - 1 if ragged else q.shape[0]
    if B < 0:
        raise ValueError("new_start must have one entry more than there are sequences")
    n, heads, dim, *q_strides = _rows(q, "q", B, ragged)
    nk, kv_heads, dk, *k_strides = _rows(k, "k", B, ragged)
    nv, hv, dv, *v_strides = _rows(v, "v", B, ragged)
    if (nk, dk) != (n, dim) or (nv, hv, dv) != (nk, kv_heads, dk) or k.shape != v.shape or not q.dtype == k.dtype == v.dtype:
        raise ValueError("q, k and v must match in tokens, dim and dtype, and k and v in heads")
    out_strides = (heads * dim, dim)
    if out is not None:
        if out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must match q in shape and dtype")
        _, _, _, *out_strides = _rows(out, "out", B, ragged)
    _int32(status, "row_status", B, _PER_SEQUENCE)
    most = _new(start, max_new, q, B)
    # (of packed rows no sequence has more than there are; the library refuses bounds whose rows of heads pass 32 bits)
    a = N.PromptAttentionDesc(B, heads, kv_heads, dim, min(most, n) if ragged else most, n, _code(q), dim ** -0.5 if scale is None else scale,
                              _count(window, "window"), _count(sinks, "sinks"), *q_strides, *k_strides, *v_strides, *out_strides)
    return ctypes.byref(a), _one_device(q, k, v, start, out, status)


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, new_start: torch.Tensor | None = None,
                     max_new: int | None = None, scale: float | None = None, window: int = 0, sinks: int = 0, lse: bool = False,
                     out: torch.Tensor | None = None, row_status: torch.Tensor | None = None, stream=None):
    """Causal attention of whole prompts over their own keys and values; see
    sv_prompt_attention.

    q [B, n, heads, dim], k and v [B, n, kv_heads, dim] (or [total, ...] with
    ``new_start`` [B + 1] and ``max_new``, the most tokens of a sequence),
    float32 or bfloat16; ``scale`` defaults to 1 / sqrt(dim).  Returns out like
    q, and with ``lse`` the log-sum-exp [..., heads] float32 as well.

    Rows of no sequence, and of sequences that are left out (``row_status``
    says which), are not written: in ``out`` they keep what they had, in results
    that the call makes itself they hold anything."""
    a, gpu = _prompt_plan(_meta(q), _meta(k), _meta(v), _meta(new_start), None if max_new is None else int(max_new),
                          None if scale is None else float(scale), int(window), int(sinks), _meta(out), _meta(row_status))
    if out is None:
        out = _empty_like(q, stream)
    sums = _empty(q.shape[:-1], torch.float32, q.device, stream) if lse else None
    _call(gpu, "sv_prompt_attention", a, q.data_ptr(), k.data_ptr(), v.data_ptr(), _at(new_start), out.data_ptr(), _at(sums),
          _at(row_status), _stream_of(stream, gpu))
    return (out, sums) if lse else out
