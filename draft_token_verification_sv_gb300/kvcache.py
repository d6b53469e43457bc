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

A call's checks and descriptors depend on the tensors' shapes, strides and
types alone, so they are made once for each combination and kept (what a call
costs on the host is most of a decoding step's small launches).
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native as N
from .verify import _WORKSPACES, _code, workspace

_CODES = (torch.float8_e4m3fn, torch.uint8)
_KEPT = 4096  # combinations of shapes kept for each entry point

_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def kv_cache(num_pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda") -> dict:
    """An empty cache of one layer (codes 0, scales 1)."""
    def codes():
        return torch.zeros((num_pages, kv_heads, page_size, head_dim), dtype=torch.uint8,
                           device=device).view(torch.float8_e4m3fn)

    def scales():
        return torch.ones((num_pages, kv_heads), dtype=torch.float32, device=device)
    return dict(k=codes(), v=codes(), k_scale=scales(), v_scale=scales())


def kv_pool(num_pages: int, device="cuda") -> dict:
    """The free pages of a cache, all of them: ``free``, a stack of page ids
    (page 0 on top), and ``count``, how many are on it."""
    return dict(free=torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device),
                count=torch.full((1,), num_pages, dtype=torch.int32, device=device))


class _Meta(tuple):
    """What the checks see of a tensor: (shape, strides, dtype, GPU or -1)."""
    __slots__ = ()
    shape = property(lambda m: m[0])
    strides = property(lambda m: m[1])
    dtype = property(lambda m: m[2])
    device = property(lambda m: m[3])


def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _see(meta, name) -> _Meta:
    if meta is None:
        return None
    m = _Meta(meta)
    if m.device < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return m


def _one_device(*metas) -> int:
    devices = {m[3] for m in metas if m is not None}
    if len(devices) > 1:
        raise ValueError("all tensors of a call must be on one GPU")
    return devices.pop()


def _numel(shape) -> int:
    n = 1
    for x in shape:
        n *= x
    return n


def _count(n: int, name: str) -> int:
    """``n``, if the descriptors' 32 bits hold it."""
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, got {n}")
    return n


def _contiguous(m: _Meta) -> bool:
    want = 1
    for n, s in zip(reversed(m.shape), reversed(m.strides)):
        if n != 1 and s != want and _numel(m.shape) > 0:
            return False
        want *= n
    return True


def _int32(meta, name, numel, what):
    m = _see(meta, name)
    if m is None:
        return
    if m.dtype != torch.int32 or not _contiguous(m):
        raise ValueError(f"{name} must be a contiguous int32 tensor")
    if _numel(m.shape) != numel:
        raise ValueError(f"{name} must have {what}")


def _table(table: _Meta):
    """(sequences, columns, row stride) of a page table."""
    if table.dtype != torch.int32 or len(table.shape) != 2 or table.strides[1] != 1 and table.shape[1] > 1:
        raise ValueError("page_table must be an int32 [B, pages] tensor with contiguous rows")
    B, columns = table.shape
    if B > 1 and table.strides[0] < columns:
        raise ValueError("page_table rows overlap in memory (an expanded tensor? .contiguous() gives every sequence a row)")
    return B, columns, table.strides[0] if B > 1 else columns


def _kv_desc(k, v, ks, vs, table, lens, name) -> N.KvDesc:
    k, v, ks, vs = _see(k, "cache['k']"), _see(v, "cache['v']"), _see(ks, "cache['k_scale']"), _see(vs, "cache['v_scale']")
    table = _see(table, "page_table")
    if k.dtype not in _CODES or v.dtype not in _CODES:
        raise TypeError("cache codes must be float8_e4m3fn or uint8")
    if len(k.shape) != 4 or k.shape != v.shape or k.strides != v.strides or k.strides[3] != 1:
        raise ValueError("cache['k'] and cache['v'] must be [pages, kv_heads, page_size, head_dim] with the same "
                         "strides and a contiguous last dimension")
    for m, n in ((ks, "cache['k_scale']"), (vs, "cache['v_scale']")):
        if m.dtype != torch.float32 or m.shape != k.shape[:2] or not _contiguous(m):
            raise ValueError(f"{n} must be a contiguous float32 [pages, kv_heads] tensor")
    B, columns, table_stride = _table(table)
    _int32(lens, name, B, "one entry for each row of page_table")
    pages, heads, page, dim = k.shape
    # a dimension of one entry is never stepped over: its stride may be anything
    step = [s if n > 1 else -(-max(s, dim) // 16) * 16 for n, s in zip(k.shape[:3], k.strides)]
    return N.KvDesc(B, heads, dim, page, pages, columns, step[0], step[1], step[2],
                    table_stride)


def _rows(m: _Meta, name: str, B: int, ragged: bool):
    """(rows, heads, dim, row stride, head stride) of [B, n, heads, dim] or [total, heads, dim]."""
    shape, strides = m.shape, m.strides
    if len(shape) != (3 if ragged else 4):
        raise ValueError(f"{name} must be [total, heads, dim] with new_start, else [B, n, heads, dim]")
    heads, dim = shape[-2:]
    _count(_numel(shape[:-2]), f"the number of {name}'s rows")
    if strides[-1] != 1:
        raise ValueError(f"{name}: last dimension must be contiguous")
    head_stride = strides[-2] if heads > 1 else dim
    if ragged:
        return shape[0], heads, dim, strides[0] if shape[0] > 1 else max(dim, strides[0]), head_stride
    if shape[0] != B:
        raise ValueError(f"{name} must have one entry for each row of page_table")
    n = shape[1]
    row_stride = strides[1] if n > 1 else strides[0]
    if B > 1 and n > 1 and strides[0] != n * strides[1]:
        raise ValueError(f"{name}: rows are not evenly spaced")
    return B * n, heads, dim, row_stride if B * n > 1 else max(dim, row_stride), head_stride


def _new(new_start, max_new, m: _Meta, B):
    """max_new of a call whose new tokens have the shape of ``m``."""
    if new_start is None:
        if max_new is not None and len(m.shape) == 4 and max_new != m.shape[1]:
            raise ValueError("max_new differs from the tokens given")
        return m.shape[1] if len(m.shape) == 4 else 0
    _int32(new_start, "new_start", B + 1, "one entry more than page_table has rows")
    if max_new is None:
        raise ValueError("new_start needs max_new, the largest number of new tokens of a sequence")
    return _count(max_new, "the largest number of new tokens")


_PER_SEQUENCE = "one entry for each sequence"


@functools.lru_cache(maxsize=_KEPT)
def _append_plan(kc, vc, ks, vs, table, lens, k, v, start, max_new, status):
    d = _kv_desc(kc, vc, ks, vs, table, lens, "ctx_lens")
    k, v = _see(k, "k"), _see(v, "v")
    B, ragged = d.batch, start is not None
    n, hk, dk, k_row, k_head = _rows(k, "k", B, ragged)
    nv, hv, dv, v_row, v_head = _rows(v, "v", B, ragged)
    if (n, hk, dk) != (nv, hv, dv) or k.dtype != v.dtype:
        raise ValueError("k and v must match in shape and dtype")
    if hk != d.kv_heads or dk != d.head_dim:
        raise ValueError("k and v must have the cache's heads and head_dim")
    r = N.KvRowsDesc(_new(start, max_new, k, B), n, _code(k), 0, k_row, k_head, v_row, v_head)
    _int32(status, "row_status", B, _PER_SEQUENCE)
    return ctypes.byref(d), ctypes.byref(r), _one_device(kc, vc, ks, vs, table, lens, k, v, start, status)


@functools.lru_cache(maxsize=_KEPT)
def _read_plan(kc, vc, ks, vs, table, first, k, v, start, tokens, status):
    d = _kv_desc(kc, vc, ks, vs, table, first, "first")
    k, v = _see(k, "out[0]"), _see(v, "out[1]")
    B, ragged = d.batch, start is not None
    for m, name in ((k, "out[0]"), (v, "out[1]")):
        if m.shape != k.shape or m.dtype != k.dtype or tuple(m.shape[-2:]) != (d.kv_heads, d.head_dim):
            raise ValueError(f"{name} must be [..., {d.kv_heads}, {d.head_dim}], both of one shape and dtype")
    n, _, _, k_row, k_head = _rows(k, "out[0]", B, ragged)
    _, _, _, v_row, v_head = _rows(v, "out[1]", B, ragged)
    r = N.KvRowsDesc(_new(start, tokens, k, B), n, _code(k), 0, k_row, k_head, v_row, v_head)
    _int32(status, "row_status", B, _PER_SEQUENCE)
    return ctypes.byref(d), ctypes.byref(r), _one_device(kc, vc, ks, vs, table, first, k, v, start, status)


@functools.lru_cache(maxsize=_KEPT)
def _commit_plan(kc, vc, ks, vs, table, lens, path, accept, new_lens, status):
    d = _kv_desc(kc, vc, ks, vs, table, lens, "ctx_lens")
    B, p = d.batch, _see(path, "path")
    if len(p.shape) != 2:
        raise ValueError("path must be [B, D+1]")
    _int32(path, "path", B * p.shape[1], "one row for each sequence")
    _int32(accept, "accept_len", B, _PER_SEQUENCE)
    _int32(new_lens, "new_lens", B, _PER_SEQUENCE)
    _int32(status, "row_status", B, _PER_SEQUENCE)
    return ctypes.byref(d), p.shape[1], _one_device(kc, vc, ks, vs, table, lens, path, accept, new_lens, status)


@functools.lru_cache(maxsize=_KEPT)
def _attention_plan(q, kc, vc, ks, vs, table, lens, start, max_new, parents, scale, window, sinks, out, status):
    d = _kv_desc(kc, vc, ks, vs, table, lens, "ctx_lens")
    q, out = _see(q, "q"), _see(out, "out")
    B, ragged = d.batch, start is not None
    n, heads, dim, q_row, q_head = _rows(q, "q", B, ragged)
    if dim != d.head_dim:
        raise ValueError("q must have the cache's head_dim")
    _int32(parents, "parents", n, "one entry for each new token")
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q in shape and dtype")
    _, _, _, o_row, o_head = _rows(out, "out", B, ragged)
    a = N.KvAttentionDesc(d, heads, _new(start, max_new, q, B), n, _code(q),
                          dim ** -0.5 if scale is None else scale, _count(window, "window"), _count(sinks, "sinks"), 0, q_row, q_head,
                          o_row, o_head)
    _int32(status, "row_status", B, _PER_SEQUENCE)
    return (ctypes.byref(a), N.lib().sv_kv_attention_workspace_size(ctypes.byref(a)),
            _one_device(kc, vc, ks, vs, table, lens, q, start, parents, out, status))


@functools.lru_cache(maxsize=_KEPT)
def _assign_plan(free, count, table, held, lens, page, start, max_new, total, parents, slots, positions, status):
    """slots and positions None: the call makes its results itself, or has none."""
    free, count, table = _see(free, "pool['free']"), _see(count, "pool['count']"), _see(table, "page_table")
    if free.dtype != torch.int32 or len(free.shape) != 1 or not _contiguous(free):
        raise ValueError("pool['free'] must be a contiguous int32 [num_pages] tensor")
    _int32(count, "pool['count']", 1, "one entry")
    B, columns, stride = _table(table)
    _int32(held, "held", B, "one entry for each row of page_table")
    _int32(lens, "ctx_lens", B, "one entry for each row of page_table")
    _int32(status, "row_status", B, _PER_SEQUENCE)
    if start is not None:
        _int32(start, "new_start", B + 1, "one entry more than page_table has rows")
    if slots is not None:
        s, p = _see(slots, "slots"), _see(positions, "positions")
        if s.dtype != torch.int64 or not _contiguous(s) or p.dtype != torch.int32 or not _contiguous(p) or p.shape != s.shape:
            raise ValueError("slots must be a contiguous int64 tensor and positions a contiguous int32 tensor of its shape")
        if total is None:
            total = _numel(s.shape)
        elif total != _numel(s.shape):
            raise ValueError("total differs from the results given")
    if start is None:
        if total not in (None, B * max_new):
            raise ValueError("slots and positions must have one entry for each new token")
        total = B * max_new
    elif total is None:
        raise ValueError("new_start needs total, the number of rows")
    _count(max_new, "the largest number of new tokens")
    _count(total, "the number of new tokens")
    if max_new < 0 or total < 0:
        raise ValueError("there cannot be fewer than no new tokens")
    _int32(parents, "parents", total, "one entry for each new token")
    d = N.KvAssignDesc(B, _count(page, "page_size"), _count(free.shape[0], "the number of pages"), columns, max_new, total, stride)
    return ctypes.byref(d), (total,) if start is not None else (B, max_new), _one_device(free, count, table, held, lens, start, parents, slots,
                                                                                       positions, status)


def _at(t):
    return None if t is None else t.data_ptr()


def _stream_of(stream, device: int) -> int:
    if stream is None:
        return _raw_stream(device)
    if stream.device_index != device:
        raise ValueError("stream belongs to another GPU than the tensors")
    return stream.cuda_stream


def _call(device: int, entry: str, *args) -> None:
    """A call of the library with its tensors' GPU as the current one."""
    if _current_device() == device:
        st = getattr(N.lib(), entry)(*args)
    else:
        with torch.cuda.device(device):
            st = getattr(N.lib(), entry)(*args)
    if st:
        N.check(st, entry)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A result that a call on ``stream`` writes and the current stream may
    use: allocated on the one, so that no earlier use of its memory is still
    under way there, and released behind the other."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def kv_assign(pool: dict, page_table: torch.Tensor, held: torch.Tensor, ctx_lens: torch.Tensor, page_size: int, *,
              new_start: torch.Tensor | None = None, max_new: int = 0, total: int | None = None,
              parents: torch.Tensor | None = None, out: tuple | None = None, row_status: torch.Tensor | None = None,
              stream=None) -> dict:
    """Make every sequence hold the pages that its cached and ``max_new`` new
    tokens need, from and to ``pool`` (see kv_pool), and say where the new ones
    go; see sv_kv_assign.  ``held`` [B] int32 counts the entries of each
    page_table row that the sequence holds.  With ``new_start`` [B + 1] each
    sequence has its own number of new tokens, ``max_new`` at most and
    ``total`` in all; ``parents`` makes them trees.  Without new tokens, pages
    beyond ctx_lens go back.

    Updates pool, page_table and held, and returns dict(slots=int64,
    positions=int32), each [B, max_new] or [total] (or ``out``, the two); both
    are None where ``max_new`` is 0.  Rows of no sequence, and of those whose
    starts are no rows of the call, are not written: in results that the call
    makes itself they hold anything."""
    max_new = int(max_new)
    slots, positions = (None, None) if out is None else out
    if out is not None and (slots is None or positions is None):
        raise ValueError("out must be (slots, positions), both of them")
    free, count = pool["free"], pool["count"]
    d, shape, gpu = _assign_plan(_meta(free), _meta(count), _meta(page_table), _meta(held), _meta(ctx_lens), int(page_size),
                                 _meta(new_start), max_new, None if total is None else int(total), _meta(parents), _meta(slots),
                                 _meta(positions), _meta(row_status))
    if out is None and max_new > 0:
        device = ctx_lens.device
        slots, positions = _empty(shape, torch.int64, device, stream), _empty(shape, torch.int32, device, stream)
    _call(gpu, "sv_kv_assign", d, free.data_ptr(), count.data_ptr(), page_table.data_ptr(), held.data_ptr(), ctx_lens.data_ptr(),
          _at(new_start), _at(parents), _at(slots) or None, _at(positions) or None, _at(row_status), _stream_of(stream, gpu))
    return dict(slots=slots, positions=positions)


def kv_append(cache: dict, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, ctx_lens: torch.Tensor, *,
              new_start: torch.Tensor | None = None, max_new: int | None = None,
              row_status: torch.Tensor | None = None, stream=None) -> dict:
    """Quantise the new tokens' keys and values behind the cached ones; see
    sv_kv_append.  k, v [B, n, kv_heads, dim] (or [total, kv_heads, dim] with
    ``new_start``), float32 or bfloat16, any row and head strides.  Updates
    and returns ``cache``; ``row_status`` [B] int32 receives the flags."""
    kc, vc, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    d, r, gpu = _append_plan(_meta(kc), _meta(vc), _meta(ks), _meta(vs), _meta(page_table), _meta(ctx_lens), _meta(k), _meta(v),
                             _meta(new_start), None if max_new is None else int(max_new), _meta(row_status))
    _call(gpu, "sv_kv_append", d, r, k.data_ptr(), v.data_ptr(), page_table.data_ptr(), ctx_lens.data_ptr(), _at(new_start),
          kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(), _at(row_status), _stream_of(stream, gpu))
    return cache


def kv_read(cache: dict, page_table: torch.Tensor, first: torch.Tensor, tokens: int, *,
            new_start: torch.Tensor | None = None, total: int | None = None, dtype: torch.dtype = torch.bfloat16,
            out: tuple | None = None, row_status: torch.Tensor | None = None, stream=None):
    """Read tokens first[b] .. of every sequence back; see sv_kv_read.

    Returns (k, v): [B, tokens, kv_heads, dim], or with ``new_start`` [B + 1]
    [total, kv_heads, dim] rows, ``tokens`` being the most of one sequence."""
    kc, vc, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    tokens = int(tokens)
    if out is None:
        _, heads, _, dim = kc.shape
        if new_start is None:
            shape = (page_table.shape[0], tokens, heads, dim)
        elif total is None:
            raise ValueError("new_start needs total, the number of rows")
        else:
            shape = (int(total), heads, dim)
        k, v = _empty(shape, dtype, kc.device, stream), _empty(shape, dtype, kc.device, stream)
    else:
        k, v = out
    d, r, gpu = _read_plan(_meta(kc), _meta(vc), _meta(ks), _meta(vs), _meta(page_table), _meta(first), _meta(k), _meta(v),
                           _meta(new_start), tokens, _meta(row_status))
    _call(gpu, "sv_kv_read", d, r, kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(), page_table.data_ptr(),
          first.data_ptr(), _at(new_start), k.data_ptr(), v.data_ptr(), _at(row_status), _stream_of(stream, gpu))
    return k, v


def kv_commit(cache: dict, page_table: torch.Tensor, ctx_lens: torch.Tensor, path: torch.Tensor,
              accept_len: torch.Tensor, nodes: int, *, new_lens: torch.Tensor | None = None,
              row_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Keep the accepted path of a scored tree of ``nodes`` tokens; see
    sv_kv_commit.  path [B, D+1] and accept_len [B] int32 are the results of
    verify_tree or verify_tree_sample.  Returns the sequences' new lengths
    [B] int32 and updates ``cache``."""
    kc, vc, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    if new_lens is None:
        new_lens = _empty(ctx_lens.shape, ctx_lens.dtype, ctx_lens.device, stream)
    d, length, gpu = _commit_plan(_meta(kc), _meta(vc), _meta(ks), _meta(vs), _meta(page_table), _meta(ctx_lens), _meta(path),
                                  _meta(accept_len), _meta(new_lens), _meta(row_status))
    _call(gpu, "sv_kv_commit", d, _count(int(nodes), "nodes"), length, page_table.data_ptr(), ctx_lens.data_ptr(), path.data_ptr(),
          accept_len.data_ptr(), kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(), new_lens.data_ptr(),
          _at(row_status), _stream_of(stream, gpu))
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
    kc, vc, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    device = q.device
    if out is None:
        out = _empty(q.shape, q.dtype, device, stream)
    a, need, gpu = _attention_plan(_meta(q), _meta(kc), _meta(vc), _meta(ks), _meta(vs), _meta(page_table), _meta(ctx_lens),
                                   _meta(new_start), None if max_new is None else int(max_new), _meta(parents),
                                   None if scale is None else float(scale), int(window), int(sinks),
                                   _meta(out), _meta(row_status))
    sums = _empty(q.shape[:-1], torch.float32, device, stream) if lse else None
    raw = _stream_of(stream, gpu)
    if ws is None:
        ws = _WORKSPACES.get((gpu, raw))
        if ws is None or ws.numel() < need:
            ws = workspace(need, device, stream)
    elif ws.get_device() != gpu or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous tensor on the GPU of the other tensors")
    _call(gpu, "sv_kv_attention", a, q.data_ptr(), kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(),
          page_table.data_ptr(), ctx_lens.data_ptr(), _at(new_start), _at(parents), out.data_ptr(), _at(sums),
          _at(row_status), ws.data_ptr(), ws.numel(), raw)
    return (out, sums) if lse else out
