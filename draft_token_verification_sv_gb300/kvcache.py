"""PyTorch-facing wrappers of the target's 8-bit cache and the attention over
it (argument marshalling only; see the cache section of include/spec_verify.h).

A cache is a dict of four tensors of one layer, as ``kv_cache`` makes it:
``k`` and ``v`` [num_pages, kv_heads, page_size, head_dim] e4m3 codes
(float8_e4m3fn or uint8; any strides that are multiples of 16 with the last
dimension contiguous, the same for both, so a [num_pages, page_size,
kv_heads, head_dim] array transposed is as good) and ``k_scale``, ``v_scale``
[num_pages, kv_heads] float32.

New tokens come as [B, n, ...] tensors (every sequence has n) or, with
``new_start`` [B + 1] int32 and ``max_new``, as [total, ...] rows.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native as N
from .verify import _code, _cuda, _i32, _p, _stream, workspace

_CODES = (torch.float8_e4m3fn, torch.uint8)


def kv_cache(num_pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda") -> dict:
    """An empty cache of one layer (codes 0, scales 1)."""
    def codes():
        return torch.zeros((num_pages, kv_heads, page_size, head_dim), dtype=torch.uint8,
                           device=device).view(torch.float8_e4m3fn)

    def scales():
        return torch.ones((num_pages, kv_heads), dtype=torch.float32, device=device)
    return dict(k=codes(), v=codes(), k_scale=scales(), v_scale=scales())


@functools.lru_cache(maxsize=1024)
def _kv_desc(shape, stride, batch, columns, table_stride) -> N.KvDesc:
    pages, heads, page, dim = shape
    # a dimension of one entry is never stepped over: its stride may be anything
    step = [s if n > 1 else -(-max(s, dim) // 16) * 16 for n, s in zip(shape[:3], stride)]
    return N.KvDesc(batch, heads, dim, page, pages, columns, step[0], step[1], step[2], max(table_stride, columns))


def _cache(cache, page_table, lens, name) -> N.KvDesc:
    k, v, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    for t, n in ((k, "cache['k']"), (v, "cache['v']"), (ks, "cache['k_scale']"), (vs, "cache['v_scale']"),
                 (page_table, "page_table"), (lens, name)):
        _cuda(t, n)
    if k.dtype not in _CODES or v.dtype not in _CODES:
        raise TypeError("cache codes must be float8_e4m3fn or uint8")
    if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1:
        raise ValueError("cache['k'] and cache['v'] must be [pages, kv_heads, page_size, head_dim] with the same "
                         "strides and a contiguous last dimension")
    for t, n in ((ks, "cache['k_scale']"), (vs, "cache['v_scale']")):
        if t.dtype != torch.float32 or t.shape != k.shape[:2] or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous float32 [pages, kv_heads] tensor")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.stride(1) != 1 and page_table.shape[1] > 1:
        raise ValueError("page_table must be an int32 [B, pages] tensor with contiguous rows")
    _i32(lens, name)
    B, columns = page_table.shape
    if lens.numel() != B:
        raise ValueError(f"{name} must have one entry for each row of page_table")
    return _kv_desc(k.shape, k.stride(), B, columns, page_table.stride(0) if B > 1 else columns)


def _status(row_status, B):
    _cuda(row_status, "row_status")
    if row_status is not None and _i32(row_status, "row_status").numel() != B:
        raise ValueError("row_status must have one entry for each sequence")
    return _p(row_status)


def _rows(t: torch.Tensor, name: str, B: int, ragged: bool):
    """(rows, heads, dim, row stride, head stride) of [B, n, heads, dim] or [total, heads, dim]."""
    if t.dim() != (3 if ragged else 4):
        raise ValueError(f"{name} must be [total, heads, dim] with new_start, else [B, n, heads, dim]")
    shape, stride = t.shape, t.stride()
    heads, dim = shape[-2:]
    if stride[-1] != 1:
        raise ValueError(f"{name}: last dimension must be contiguous")
    head_stride = stride[-2] if heads > 1 else dim
    if ragged:
        return shape[0], heads, dim, stride[0] if shape[0] > 1 else max(dim, stride[0]), head_stride
    if shape[0] != B:
        raise ValueError(f"{name} must have one entry for each row of page_table")
    n = shape[1]
    row_stride = stride[1] if n > 1 else stride[0]
    if B > 1 and n > 1 and stride[0] != n * stride[1]:
        raise ValueError(f"{name}: rows are not evenly spaced")
    return B * n, heads, dim, row_stride if B * n > 1 else max(dim, row_stride), head_stride


def _new(new_start, max_new, t, name, B):
    """max_new of a call whose new tokens are ``t``."""
    if new_start is None:
        if max_new is not None and t.dim() == 4 and max_new != t.shape[1]:
            raise ValueError("max_new differs from the tokens given")
        return t.shape[1] if t.dim() == 4 else 0
    _cuda(new_start, "new_start")
    if _i32(new_start, "new_start").numel() != B + 1:
        raise ValueError("new_start must have one entry more than page_table has rows")
    if max_new is None:
        raise ValueError("new_start needs max_new, the largest number of new tokens of a sequence")
    return int(max_new)


def kv_append(cache: dict, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, ctx_lens: torch.Tensor, *,
              new_start: torch.Tensor | None = None, max_new: int | None = None,
              row_status: torch.Tensor | None = None, stream=None) -> dict:
    """Quantise the new tokens' keys and values behind the cached ones; see
    sv_kv_append.  k, v [B, n, kv_heads, dim] (or [total, kv_heads, dim] with
    ``new_start``), float32 or bfloat16, any row and head strides.  Updates
    and returns ``cache``; ``row_status`` [B] int32 receives the flags."""
    d = _cache(cache, page_table, ctx_lens, "ctx_lens")
    _cuda(k, "k")
    _cuda(v, "v")
    B = d.batch
    ragged = new_start is not None
    n, hk, dk, k_row, k_head = _rows(k, "k", B, ragged)
    nv, hv, dv, v_row, v_head = _rows(v, "v", B, ragged)
    if (n, hk, dk) != (nv, hv, dv) or k.dtype != v.dtype:
        raise ValueError("k and v must match in shape and dtype")
    if hk != d.kv_heads or dk != d.head_dim:
        raise ValueError("k and v must have the cache's heads and head_dim")
    r = N.KvRowsDesc(_new(new_start, max_new, k, "k", B), n, _code(k), 0, k_row, k_head, v_row, v_head)
    st = N.lib().sv_kv_append(
        ctypes.byref(d), ctypes.byref(r), _p(k), _p(v), _p(page_table), _p(ctx_lens), _p(new_start), _p(cache["k"]),
        _p(cache["v"]), _p(cache["k_scale"]), _p(cache["v_scale"]), _status(row_status, B), _stream(stream))
    N.check(st, "sv_kv_append")
    return cache


def kv_read(cache: dict, page_table: torch.Tensor, first: torch.Tensor, tokens: int, *,
            new_start: torch.Tensor | None = None, total: int | None = None, dtype: torch.dtype = torch.bfloat16,
            out: tuple | None = None, row_status: torch.Tensor | None = None, stream=None):
    """Read tokens first[b] .. of every sequence back; see sv_kv_read.

    Returns (k, v): [B, tokens, kv_heads, dim], or with ``new_start`` [B + 1]
    [total, kv_heads, dim] rows, ``tokens`` being the most of one sequence."""
    d = _cache(cache, page_table, first, "first")
    B = d.batch
    if new_start is None:
        shape = (B, int(tokens), d.kv_heads, d.head_dim)
    else:
        if total is None:
            raise ValueError("new_start needs total, the number of rows")
        shape = (int(total), d.kv_heads, d.head_dim)
    if out is None:
        out = tuple(torch.empty(shape, dtype=dtype, device=cache["k"].device) for _ in range(2))
    k, v = out
    for t, n in ((k, "out[0]"), (v, "out[1]")):
        _cuda(t, n)
        if tuple(t.shape) != shape or t.dtype != k.dtype:
            raise ValueError(f"{n} must be {list(shape)}, both of one dtype")
    ragged = new_start is not None
    n, _, _, k_row, k_head = _rows(k, "out[0]", B, ragged)
    _, _, _, v_row, v_head = _rows(v, "out[1]", B, ragged)
    r = N.KvRowsDesc(_new(new_start, int(tokens), k, "out[0]", B), n, _code(k), 0, k_row, k_head, v_row, v_head)
    st = N.lib().sv_kv_read(
        ctypes.byref(d), ctypes.byref(r), _p(cache["k"]), _p(cache["v"]), _p(cache["k_scale"]), _p(cache["v_scale"]),
        _p(page_table), _p(first), _p(new_start), _p(k), _p(v), _status(row_status, B), _stream(stream))
    N.check(st, "sv_kv_read")
    return k, v


def kv_commit(cache: dict, page_table: torch.Tensor, ctx_lens: torch.Tensor, path: torch.Tensor,
              accept_len: torch.Tensor, nodes: int, *, new_lens: torch.Tensor | None = None,
              row_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Keep the accepted path of a scored tree of ``nodes`` tokens; see
    sv_kv_commit.  path [B, D+1] and accept_len [B] int32 are the results of
    verify_tree or verify_tree_sample.  Returns the sequences' new lengths
    [B] int32 and updates ``cache``."""
    d = _cache(cache, page_table, ctx_lens, "ctx_lens")
    _cuda(path, "path")
    _cuda(accept_len, "accept_len")
    B = d.batch
    if _i32(path, "path").dim() != 2 or path.shape[0] != B or _i32(accept_len, "accept_len").numel() != B:
        raise ValueError("path must be [B, D+1] and accept_len [B]")
    if new_lens is None:
        new_lens = torch.empty(B, dtype=torch.int32, device=path.device)
    _cuda(new_lens, "new_lens")
    if _i32(new_lens, "new_lens").numel() != B:
        raise ValueError("new_lens must have one entry for each sequence")
    st = N.lib().sv_kv_commit(
        ctypes.byref(d), int(nodes), path.shape[1], _p(page_table), _p(ctx_lens), _p(path), _p(accept_len),
        _p(cache["k"]), _p(cache["v"]), _p(cache["k_scale"]), _p(cache["v_scale"]), _p(new_lens),
        _status(row_status, B), _stream(stream))
    N.check(st, "sv_kv_commit")
    return new_lens


def kv_attention(q: torch.Tensor, cache: dict, page_table: torch.Tensor, ctx_lens: torch.Tensor, *,
                 new_start: torch.Tensor | None = None, max_new: int | None = None,
                 parents: torch.Tensor | None = None, scale: float | None = None, window: int = 0, sinks: int = 0,
                 lse: bool = False, out: torch.Tensor | None = None, row_status: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None, stream=None):
    """Attention of the new tokens' queries over the cache, which already
    holds their keys and values; see sv_kv_attention.

    q [B, n, heads, dim] (or [total, heads, dim] with ``new_start``), float32
    or bfloat16; ``parents`` ([B, n] or [total] int32) makes the new tokens a
    tree; ``scale`` defaults to 1 / sqrt(dim).  Returns out like q, and with
    ``lse`` the log-sum-exp [..., heads] float32 as well."""
    d = _cache(cache, page_table, ctx_lens, "ctx_lens")
    _cuda(q, "q")
    _cuda(parents, "parents")
    B = d.batch
    ragged = new_start is not None
    n, heads, dim, q_row, q_head = _rows(q, "q", B, ragged)
    if dim != d.head_dim:
        raise ValueError("q must have the cache's head_dim")
    if parents is not None and _i32(parents, "parents").numel() != n:
        raise ValueError("parents must have one entry for each new token")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    _cuda(out, "out")
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q in shape and dtype")
    _, _, _, o_row, o_head = _rows(out, "out", B, ragged)
    sums = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if lse else None
    a = N.KvAttentionDesc(d, heads, _new(new_start, max_new, q, "q", B), n, _code(q),
                          float(scale) if scale is not None else dim ** -0.5, int(window), int(sinks), 0, q_row, q_head,
                          o_row, o_head)
    lib = N.lib()
    need = lib.sv_kv_attention_workspace_size(ctypes.byref(a))
    if ws is None:
        ws = workspace(need, q.device, stream)
    st = lib.sv_kv_attention(
        ctypes.byref(a), _p(q), _p(cache["k"]), _p(cache["v"]), _p(cache["k_scale"]), _p(cache["v_scale"]),
        _p(page_table), _p(ctx_lens), _p(new_start), _p(parents), _p(out), _p(sums), _status(row_status, B), _p(ws),
        ctypes.c_size_t(ws.numel()), _stream(stream))
    N.check(st, "sv_kv_attention")
    return (out, sums) if lse else out
