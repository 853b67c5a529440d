"""A key/value cache in pages: decoding over it, writing into it, and keeping it.

``PagedKV`` wraps the K and V pools; the functions here take it with a block
table, the rows' lengths and the pages' reference counts (int32 CUDA tensors)
and call the C ABI (include/fa.h states each call's rules).  Nothing
synchronises or copies to the host.  Outputs are allocated with torch on the
stream that the call runs on; all tensors live on the current CUDA device.

A serving loop::

    cache = PagedKV(k_pool, v_pool)            # [layers, pages, h_kv, page_size, d]
    table, kv_len, ref = cache.empty(rows=64, max_pages=512)
    new_len, ref, info = reserve(cache, table, kv_len, ref, n_new)
    for layer in range(cache.num_layers):
        append(k_new, v_new, cache, layer, table, kv_len, new_len)
        o, lse = decode(q, cache, layer, table, new_len, window=(4095, 0), sinks=4)
    kv_len = new_len
    table, ref = trim(cache, table, kv_len, ref, 4095, 4)
    table, kv_len, ref, info = fork(cache, table, kv_len, ref, parent)
"""
import ctypes
import math

import torch

from . import fa

_current_device = torch.cuda.current_device
# the current stream of a device as a raw handle; torch.cuda.current_stream()
# takes 3 us of the about 15 that a small call costs its host
_current_raw_stream = torch._C._cuda_getCurrentRawStream
_int32, _bf16 = torch.int32, torch.bfloat16
_count = fa.int32_count


def _on_stream(call, stream, *args, **kw):
    """call(...) with `stream` the current one, so that its outputs are
    allocated for it."""
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def _apart(shape, strides):
    """Whether no two elements share a place: taken from the smallest stride
    up, each axis steps past everything inside it."""
    extent = 1
    for stride, n in sorted((s, n) for s, n in zip(strides, shape) if n > 1):
        if stride < extent:
            return False
        extent += stride * (n - 1)
    return True


class PagedKV:
    """The K and V pools: two bf16 CUDA tensors [layers, pages, h_kv,
    page_size, d] (or [pages, h_kv, page_size, d], one layer) of the same shape
    and strides, d contiguous and the other strides multiples of 8 (a
    transposed view of [layers, pages, page_size, h_kv, d] serves as well, an
    expanded or overlapping one is refused).  Holds the tensors and the
    structure that the library reads."""

    def __init__(self, k, v):
        if k.dim() == 4:
            k, v = k[None], v[None]
        if k.dim() != 5 or k.shape != v.shape or k.dtype != torch.bfloat16 \
                or v.dtype != torch.bfloat16 or not k.is_cuda or k.device != v.device:
            raise ValueError("k, v: expected bf16 CUDA tensors [layers, pages, h_kv, page_size, "
                             "d] of one shape")
        strides = [s if n > 1 else 0 for n, s in zip(k.shape, k.stride())]
        if strides != [s if n > 1 else 0 for n, s in zip(v.shape, v.stride())]:
            raise ValueError("k, v: the strides differ")
        if k.numel() == 0:
            raise ValueError("k, v: empty pools")
        if strides[4] != 1 or any(s % 8 for s in strides[:4]):
            raise ValueError("k, v: d must be contiguous and the other strides multiples of 8")
        if not _apart(k.shape, strides):
            raise ValueError("k, v: elements share memory (an expanded or overlapping view)")
        if k.data_ptr() % 16 or v.data_ptr() % 16:
            raise ValueError("k, v: expected 16-byte aligned pools")
        self.k, self.v = k, v
        self.num_layers, self.num_pages, self.h_kv, self.page_size, self.d = k.shape
        self.device = k.device
        self.index = k.get_device()
        self.struct = fa.FaPagedKV(k.data_ptr(), v.data_ptr(), *strides[:4], self.num_layers,
                                   self.num_pages, self.page_size, self.h_kv, self.d)
        self.ref = ctypes.byref(self.struct)
        self.scale = 1.0 / math.sqrt(self.d)
        self._need = {}        # workspace sizes by a call's sizes

    def empty(self, rows, max_pages):
        """(table, kv_len, ref) of a cache without tokens."""
        ints = dict(dtype=torch.int32, device=self.device)
        return (torch.full((rows, max_pages), -1, **ints), torch.zeros(rows, **ints),
                torch.zeros(self.num_pages, **ints))


def _ints(name, t, shape, index):
    if t.dtype is not _int32 or t.shape != shape or not t.is_contiguous() \
            or t.get_device() != index:
        raise ValueError(f"{name}: expected a contiguous int32 CUDA tensor {list(shape)} on the "
                         "cache's device")
    return t.data_ptr()


def _table(cache, table):
    """The table's address and shape."""
    shape = table.shape
    if len(shape) != 2:
        raise ValueError("table: expected int32 [rows, max_pages]")
    if cache.index != _current_device():
        raise ValueError("the cache is not on the current CUDA device")
    return _ints("table", table, shape, cache.index), shape[0], shape[1]


def _check(status, where):
    if status:
        raise fa.FAError(status, where)


def _bytes(ws, need, like):
    """The address of a workspace of `need` bytes: ws, or one allocated beside
    `like` (returned to hold it)."""
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=like.device)
    elif not ws.is_cuda or not ws.is_contiguous() or ws.device != like.device:
        raise ValueError("ws: expected a contiguous CUDA tensor on the cache's device")
    elif ws.numel() * ws.element_size() < need:
        raise ValueError(f"ws: {need} bytes are needed")
    return ws, ws.data_ptr()


def _keep(cache, sizes, n):
    """n, kept under `sizes`; a cache keeps 1024 of them at most."""
    if len(cache._need) >= 1024:
        cache._need.clear()
    cache._need[sizes] = n
    return n


def _pages_need(cache, rows):
    n = cache._need.get((rows,))
    if n is None:
        n = _keep(cache, (rows,), fa.load().fa_pages_workspace_bytes(cache.num_pages, rows))
    return n


def _call_need(cache, sizes):
    """The workspace of a decode call of sizes (max_pages, rows, H, left, sinks)."""
    n = cache._need.get(sizes)
    if n is None:
        n = _keep(cache, sizes, fa.load().fa_decode_paged_call_bytes(cache.ref, *sizes))
    return n


def workspace(cache, rows=1):
    """A workspace for reserve, fork and compact of up to `rows` rows."""
    return torch.empty(_pages_need(cache, rows), dtype=torch.uint8, device=cache.device)


def decode_workspace(cache, H):
    """A workspace for decode with H query heads."""
    return torch.empty(fa.load().fa_decode_paged_workspace_bytes(H, cache.h_kv, cache.d),
                       dtype=torch.uint8, device=cache.device)


def decode(q, cache, layer, table, kv_len, scale=None, window=None, sinks=0, ws=None, stream=None):
    """(O, LSE): attention of each row's newest token (position kv_len - 1)
    over its pages; q [B, H, 1, d], O like q, LSE fp32 [B, H, 1].  window:
    (left, right), of which only left matters here, or None; sinks: first
    tokens that stay visible.  ws: decode_workspace(), else allocated
    where one is needed."""
    if stream is not None:
        return _on_stream(decode, stream, q, cache, layer, table, kv_len, scale, window, sinks, ws)
    tp, rows, max_pages = _table(cache, table)
    index = cache.index
    shape = q.shape
    if len(shape) != 4 or shape[0] != rows or shape[2] != 1 or shape[3] != cache.d \
            or q.dtype is not _bf16 or not q.is_contiguous() or q.get_device() != index:
        raise ValueError("q: expected a contiguous bf16 CUDA tensor [rows, H, 1, d]")
    lp = _ints("kv_len", kv_len, shape[:1], index)
    H = shape[1]
    left, sinks = -1 if window is None else _count(window[0]), _count(sinks)
    need = _call_need(cache, (max_pages, rows, H, left, sinks))
    o = torch.empty_like(q)
    lse = torch.empty(shape[:3], dtype=torch.float32, device=q.device)
    ws, wp = _bytes(ws, need, q) if need else (None, None)
    _check(fa.load().fa_decode_paged(
        q.data_ptr(), cache.ref, layer, tp, max_pages, lp, o.data_ptr(), lse.data_ptr(), rows, H,
        cache.scale if scale is None else scale, left, sinks, wp, need,
        _current_raw_stream(index)), "fa_decode_paged")
    return o, lse


def append(k_new, v_new, cache, layer, table, start, kv_len, stream=None):
    """Writes k_new, v_new [rows, h_kv, n, d]: token t of a row to position
    start + t where that is below kv_len."""
    if stream is not None:
        return _on_stream(append, stream, k_new, v_new, cache, layer, table, start, kv_len)
    tp, rows, max_pages = _table(cache, table)
    index = cache.index
    shape = k_new.shape
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if t.shape != shape or len(shape) != 4 or shape[0] != rows or shape[1] != cache.h_kv \
                or shape[3] != cache.d or t.dtype is not _bf16 or not t.is_contiguous() \
                or t.get_device() != index:
            raise ValueError(f"{name}: expected a contiguous bf16 CUDA tensor [rows, h_kv, n, d]")
    _check(fa.load().fa_paged_append(
        k_new.data_ptr(), v_new.data_ptr(), cache.ref, layer, tp, max_pages,
        _ints("start", start, shape[:1], index), _ints("kv_len", kv_len, shape[:1], index), rows,
        shape[2], _current_raw_stream(index)), "fa_paged_append")


def reserve(cache, table, kv_len, ref, n_new, ws=None, stream=None):
    """(kv_len, ref, info) after every row has got the pages for n_new more
    tokens; the table is updated in place.  info = [free pages left, pages that
    were missing]."""
    if stream is not None:
        return _on_stream(reserve, stream, cache, table, kv_len, ref, n_new, ws)
    tp, rows, max_pages = _table(cache, table)
    index, num_pages = cache.index, cache.num_pages
    lp = _ints("kv_len", kv_len, (rows,), index)
    ap = _ints("n_new", n_new, (rows,), index)
    rp = _ints("ref", ref, (num_pages,), index)
    need = _pages_need(cache, rows)
    len_out, ref_out = torch.empty_like(kv_len), torch.empty_like(ref)
    info = torch.empty(2, dtype=_int32, device=ref.device)
    ws, wp = _bytes(ws, need, ref)
    _check(fa.load().fa_pages_reserve(
        tp, max_pages, cache.page_size, lp, ap, rp, num_pages, rows, len_out.data_ptr(),
        ref_out.data_ptr(), info.data_ptr(), wp, need, _current_raw_stream(index)),
        "fa_pages_reserve")
    return len_out, ref_out, info


def fork(cache, table, kv_len, ref, parent, ws=None, stream=None):
    """(table, kv_len, ref, info) of the cache whose row r continues row
    parent[r] (-1: an empty row): beams are reordered, rows forked, and rows
    that nobody continues freed.  Partly filled pages that several rows
    continue are copied.  info as of reserve."""
    if stream is not None:
        return _on_stream(fork, stream, cache, table, kv_len, ref, parent, ws)
    tp, rows, max_pages = _table(cache, table)
    index = cache.index
    if parent.dim() != 1 or parent.numel() < 1:
        raise ValueError("parent: expected int32 [new rows]")
    new_rows = parent.numel()
    lp = _ints("kv_len", kv_len, (rows,), index)
    rp = _ints("ref", ref, (cache.num_pages,), index)
    pp = _ints("parent", parent, (new_rows,), index)
    need = _pages_need(cache, max(rows, new_rows))
    if new_rows == rows:
        table_out = torch.empty_like(table)
    else:
        table_out = torch.empty((new_rows, max_pages), dtype=_int32, device=ref.device)
    len_out, ref_out = torch.empty_like(parent), torch.empty_like(ref)
    info = torch.empty(2, dtype=_int32, device=ref.device)
    ws, wp = _bytes(ws, need, ref)
    _check(fa.load().fa_pages_fork(
        cache.ref, tp, max_pages, lp, rp, rows, pp, new_rows, table_out.data_ptr(),
        len_out.data_ptr(), ref_out.data_ptr(), info.data_ptr(), wp, need,
        _current_raw_stream(index)), "fa_pages_fork")
    return table_out, len_out, ref_out, info


def trim(cache, table, kv_len, ref, window_left, sinks=0, stream=None):
    """(table, ref) without the pages that no later token sees under a window
    of window_left and `sinks` first tokens."""
    if stream is not None:
        return _on_stream(trim, stream, cache, table, kv_len, ref, window_left, sinks)
    tp, rows, max_pages = _table(cache, table)
    index, num_pages = cache.index, cache.num_pages
    lp = _ints("kv_len", kv_len, (rows,), index)
    rp = _ints("ref", ref, (num_pages,), index)
    table_out, ref_out = torch.empty_like(table), torch.empty_like(ref)
    _check(fa.load().fa_pages_trim(
        tp, max_pages, cache.page_size, lp, rp, num_pages, rows, _count(window_left),
        _count(sinks), table_out.data_ptr(), ref_out.data_ptr(), _current_raw_stream(index)),
        "fa_pages_trim")
    return table_out, ref_out


def compact(cache, table, ref, ws=None, stream=None):
    """(table, ref, info) after the pages in use have moved to the front of the
    pool.  info = [pages in use, pages moved]."""
    if stream is not None:
        return _on_stream(compact, stream, cache, table, ref, ws)
    tp, rows, max_pages = _table(cache, table)
    index = cache.index
    rp = _ints("ref", ref, (cache.num_pages,), index)
    need = _pages_need(cache, rows)
    table_out, ref_out = torch.empty_like(table), torch.empty_like(ref)
    info = torch.empty(2, dtype=_int32, device=ref.device)
    ws, wp = _bytes(ws, need, ref)
    _check(fa.load().fa_pages_compact(
        cache.ref, tp, max_pages, rp, rows, table_out.data_ptr(), ref_out.data_ptr(),
        info.data_ptr(), wp, need, _current_raw_stream(index)), "fa_pages_compact")
    return table_out, ref_out, info
