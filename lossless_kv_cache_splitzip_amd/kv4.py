"""The 4-bit KV cache from torch tensors (include/splitzip.h, "4-bit KV cache").

Argument marshalling only, as in ``_native``: shapes, types and devices are
checked here, every step runs in the library.  The tensors:

* ``pages``  uint8 [n_pages, n_heads, page_bytes] (``kv4_pages`` allocates one),
  ``kv4_page_bytes(head_dim, page_tokens)`` bytes a head;
* ``table``  int32 [n_seqs, pages per sequence], ``lens`` int32 [n_seqs];
* ``cu``     int32 [n_seqs + 1], the first packed row of each sequence; None
  means one row each.  A sequence's rows stand for its last slots, and ``lens``
  counts them;
* ``mass`` float32 and ``pos`` int32 [n_pages, n_heads, page_tokens].

``max_new`` (rows of one sequence) and ``max_len`` (slots of one sequence) are
upper bounds known on the host; they default to all packed rows and to the
table's width.  Tight bounds make launches smaller.  A ``stream`` given is used
for the work and for what is allocated.  Nothing is synchronized.
"""
from __future__ import annotations

import struct

import torch

from . import _native as N

# splitzip_kv4_cache and splitzip_kv4_batch as bytes: packing them costs a third of filling a ctypes structure
_pack_cache = struct.Struct("@PIIII").pack
_pack_batch = struct.Struct("@PNPPIIII").pack
_HALF = {torch.bfloat16: N.BF16, torch.float16: N.KV4_FP16}
_ROWS = {torch.bfloat16: N.BF16, torch.float16: N.KV4_FP16, torch.float8_e5m2: N.FP8_E5M2}
_PAGE_TOKENS = {(17 * d * p // 16, d): p for d in (64, 128, 256) for p in (16, 32, 64, 128, 256)}  # by bytes a head


def kv4_page_bytes(head_dim: int, page_tokens: int) -> int:
    """Bytes of one head in one page."""
    n = int(N.load().splitzip_kv4_page_bytes(head_dim, page_tokens))
    if n == 0:
        raise N.SplitZipError(N.E_INVALID, "splitzip_kv4_page_bytes")
    return n


def kv4_pages(n_pages: int, n_heads: int, head_dim: int, page_tokens: int, device="cuda") -> torch.Tensor:
    """An empty pool of pages."""
    return torch.zeros(n_pages, n_heads, kv4_page_bytes(head_dim, page_tokens), dtype=torch.uint8, device=device)


# `dev` below is a device's index: comparing get_device() costs half of comparing devices

def _elsewhere(dev, stream):
    """The context to run in when the call is not for the current device and
    stream, else None."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"stream of {stream.device} for tensors on cuda:{dev}")
        return torch.cuda.stream(stream)
    if dev != torch._C._cuda_getDevice():  # a device tensor exists, so the runtime is up
        return torch.cuda.device(dev)
    return None


def _tensor(t, name, dtype, shape, dev):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")
    return t.data_ptr()


def _optional(t, name, dtype, shape, dev):
    return None if t is None else _tensor(t, name, dtype, shape, dev)


def _pool(pages):
    if not isinstance(pages, torch.Tensor) or not pages.is_cuda:
        raise ValueError("pages must be a device tensor")
    return pages.get_device()


def _cache(pages, head_dim):
    """(splitzip_kv4_cache, shape of the side arrays)."""
    shape = pages.shape
    if len(shape) != 3 or pages.dtype is not torch.uint8 or not pages.is_contiguous():
        raise ValueError("pages must be a contiguous uint8 tensor [n_pages, n_heads, page_bytes]")
    n, heads, size = shape
    p = _PAGE_TOKENS.get((size, head_dim))
    if p is None:
        raise ValueError(f"pages of {size} bytes a head do not hold 16 to 256 tokens of head_dim {head_dim}")
    return _pack_cache(pages.data_ptr(), n, heads, head_dim, p), (n, heads, p)


def _batch(page_tokens, table, lens, cu, n_rows, max_new, max_len, dev):
    shape = table.shape
    if len(shape) != 2 or table.dtype is not torch.int32 or table.get_device() != dev:
        raise ValueError(f"table must be an int32 tensor [n_seqs, pages] on cuda:{dev}")
    seqs, width = shape
    stride, unit = table.stride()
    if seqs <= 1:
        stride = width
    if (width > 1 and unit != 1) or stride < width:
        raise ValueError("table's rows must be contiguous and must not overlap")
    room = width * page_tokens
    if max_len is None:
        max_len = min(room, 1 << 23)
    elif not 0 <= max_len <= room:
        raise ValueError(f"max_len {max_len} exceeds the table's {width} pages of {page_tokens} tokens")
    lens_at = _tensor(lens, "lens", torch.int32, (seqs,), dev)
    cu_at = 0
    if cu is not None:
        cu_at = _tensor(cu, "cu", torch.int32, (seqs + 1,), dev)
        max_new = n_rows if max_new is None else min(max_new, n_rows)
        if max_new < (n_rows > 0):
            raise ValueError("max_new must be at least 1 where there are rows")
    else:
        if n_rows != seqs:
            raise ValueError(f"{n_rows} rows for {seqs} sequences: several rows of a sequence need cu")
        max_new = min(1, n_rows)
    return _pack_batch(table.data_ptr(), stride, lens_at, cu_at, seqs, max_len, max_new, n_rows)


def _strided(t, name, dtypes, heads, dim, dev):
    """(rows, row stride, head stride, address) of t [rows, heads, dim]."""
    shape = t.shape
    if len(shape) != 3 or t.dtype not in dtypes or t.get_device() != dev:
        raise ValueError(f"{name} must be a [rows, heads, head_dim] tensor of {' or '.join(map(str, dtypes))} on cuda:{dev}")
    rows, h, d = shape
    if d != dim or (heads is not None and h != heads):
        raise ValueError(f"{name} has shape {tuple(shape)}, heads {heads} and head_dim {dim} expected")
    s0, s1, s2 = t.stride()
    if s2 != 1:
        raise ValueError(f"{name}'s channels must be contiguous")
    if rows <= 1:
        s0 = 0
    if h <= 1:
        s1 = 0
    at = t.data_ptr()
    if (s0 | s1) & 7 or at % (8 * t.element_size()):
        raise ValueError(f"{name}'s rows and heads must start at multiples of 8 elements")
    return rows, s0, s1, at


def _check(rc, what):
    if rc != N.OK:
        raise N.SplitZipError(rc, what)


_stream = torch._C._cuda_getCurrentRawStream


def _status(status, dev):
    if status is None:
        return None
    N._status_word(status)
    if status.get_device() != dev:
        raise ValueError(f"status must be on cuda:{dev}")
    return status.data_ptr()


def _work(work, need, dev):
    if work is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    N._device_buffer(work, "work", need)
    if work.get_device() != dev:
        raise ValueError(f"work must be on cuda:{dev}")
    return work


def kv4_append(pages, k, v, table, lens, cu=None, positions=None, mass=None, pos=None, max_new=None, max_len=None,
               status=None, stream=None) -> None:
    """Put rows k, v [rows, n_heads, head_dim] (bfloat16, float16 or
    float8_e5m2, strided views allowed) into their sequences' last slots.
    ``mass`` of the slots becomes 0 and ``pos`` the rows' ``positions`` (int32
    [rows]; None: the slot's number)."""
    dev = _pool(pages)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return kv4_append(pages, k, v, table, lens, cu, positions, mass, pos, max_new, max_len, status)
    dim = k.shape[-1] if k.dim() == 3 else 0
    c, side = _cache(pages, dim)
    rows, k0, k1, k_at = _strided(k, "k", _ROWS, side[1], dim, dev)
    rows_v, v0, v1, v_at = _strided(v, "v", (k.dtype,), side[1], dim, dev)
    if rows_v != rows:
        raise ValueError(f"{rows} rows of k, {rows_v} of v")
    b = _batch(side[2], table, lens, cu, rows, max_new, max_len, dev)
    rc = N.load().splitzip_kv4_append(
        c, b, _ROWS[k.dtype], k_at, k0, k1, v_at, v0, v1,
        _optional(positions, "positions", torch.int32, (rows,), dev),
        _optional(mass, "mass", torch.float32, side, dev), _optional(pos, "pos", torch.int32, side, dev),
        _status(status, dev), _stream(dev))
    _check(rc, "splitzip_kv4_append")


def kv4_read(pages, table, lens, head_dim, cu=None, n_tokens=None, dtype=torch.bfloat16, max_new=None, max_len=None,
             out=None, status=None, stream=None):
    """(k, v) [n_tokens, n_heads, head_dim] of the sequences' last slots, the
    inverse of ``kv4_append``.  ``n_tokens``: packed rows in all (cu[-1]; the
    number of sequences where cu is None).  ``out``: the two tensors to fill;
    rows of no sequence are not written."""
    dev = _pool(pages)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return kv4_read(pages, table, lens, head_dim, cu, n_tokens, dtype, max_new, max_len, out, status)
    c, side = _cache(pages, head_dim)
    if dtype not in _HALF:
        raise ValueError("dtype must be torch.bfloat16 or torch.float16")
    if n_tokens is None:
        if cu is not None:
            raise ValueError("n_tokens is needed with cu")
        n_tokens = table.shape[0]
    shape = (n_tokens, side[1], head_dim)
    if out is None:
        k, v = torch.empty(shape, dtype=dtype, device=dev), torch.empty(shape, dtype=dtype, device=dev)
    else:
        k, v = out
        _tensor(k, "out[0]", dtype, shape, dev)
        _tensor(v, "out[1]", dtype, shape, dev)
    b = _batch(side[2], table, lens, cu, n_tokens, max_new, max_len, dev)
    rc = N.load().splitzip_kv4_read(c, b, _HALF[dtype], k.data_ptr(), v.data_ptr(), _status(status, dev),
                                    _stream(dev))
    _check(rc, "splitzip_kv4_read")
    return k, v


def kv4_attention(q, pages, table, lens, cu=None, max_new=None, scale=None, max_len=None, mass=None, mass_out=None,
                  return_lse=False, out=None, lse=None, work=None, status=None, stream=None):
    """Causal attention of packed queries q [rows, n_q_heads, head_dim]
    (bfloat16 or float16, strided views allowed) over the cache; returns
    ``out`` (contiguous, q's type), or ``(out, lse)`` with ``return_lse`` or
    ``lse`` given.  ``scale`` defaults to head_dim ** -0.5.  With ``mass``, the
    weights that every slot drew are added into ``mass_out`` (default: into
    ``mass``).  Rows of no sequence are not written."""
    dev = _pool(pages)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return kv4_attention(q, pages, table, lens, cu, max_new, scale, max_len, mass, mass_out, return_lse, out,
                                 lse, work, status)
    dim = q.shape[-1] if q.dim() == 3 else 0
    c, side = _cache(pages, dim)
    rows, q0, q1, q_at = _strided(q, "q", _HALF, None, dim, dev)
    heads = q.shape[1]
    b = _batch(side[2], table, lens, cu, rows, max_new, max_len, dev)
    if out is None:
        out = torch.empty((rows, heads, dim), dtype=q.dtype, device=dev)
    else:
        _tensor(out, "out", q.dtype, (rows, heads, dim), dev)
    if lse is not None:
        _tensor(lse, "lse", torch.float32, (rows, heads), dev)
    elif return_lse:
        lse = torch.empty((rows, heads), dtype=torch.float32, device=dev)
    mass_at = to = None
    if mass is not None:
        mass_at = to = _tensor(mass, "mass", torch.float32, side, dev)
        if mass_out is not None:
            to = _tensor(mass_out, "mass_out", torch.float32, side, dev)
    elif mass_out is not None:
        raise ValueError("mass_out needs mass")
    lib = N.load()
    need = lib.splitzip_kv4_attention_work_bytes(c, b, heads, mass is not None)
    if need == 0:
        raise N.SplitZipError(N.E_INVALID, "splitzip_kv4_attention_work_bytes")
    work = _work(work, need, dev)
    rc = lib.splitzip_kv4_attention(c, b, _HALF[q.dtype], q_at, q0, q1, heads,
                                    dim ** -0.5 if scale is None else scale, out.data_ptr(),
                                    None if lse is None else lse.data_ptr(), mass_at, to, work.data_ptr(),
                                    N._nbytes(work), _status(status, dev), _stream(dev))
    _check(rc, "splitzip_kv4_attention")
    return out if lse is None else (out, lse)


def kv4_evict(pages, table, lens, mass, pos, next_pos, head_dim, budget, sinks=0, recent=0, max_len=None,
              lens_out=None, mass_out=None, pos_out=None, work=None, status=None, stream=None):
    """Cut every sequence longer than ``budget`` slots to the ``budget`` that
    drew the largest ``mass``, each head for itself; tokens at positions below
    ``sinks`` or at ``next_pos`` - ``recent`` and beyond always stay.  Returns
    ``(lens_out, mass_out, pos_out)``, by default the tensors given, updated in
    place."""
    dev = _pool(pages)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return kv4_evict(pages, table, lens, mass, pos, next_pos, head_dim, budget, sinks, recent, max_len,
                             lens_out, mass_out, pos_out, work, status)
    c, side = _cache(pages, head_dim)
    seqs = table.shape[0]
    if min(budget, sinks, recent) < 0 or max(budget, sinks, recent) >= 1 << 32:
        raise ValueError("budget, sinks and recent must be 32-bit counts")
    lens_out = lens if lens_out is None else lens_out
    mass_out = mass if mass_out is None else mass_out
    pos_out = pos if pos_out is None else pos_out
    b = _batch(side[2], table, lens, None, seqs, 1, max_len, dev)
    lib = N.load()
    need = lib.splitzip_kv4_evict_work_bytes(c, b, budget)
    if need == 0:
        raise N.SplitZipError(N.E_INVALID, "splitzip_kv4_evict_work_bytes")
    work = _work(work, need, dev)
    rc = lib.splitzip_kv4_evict(
        c, b, budget, sinks, recent, _tensor(next_pos, "next_pos", torch.int32, (seqs,), dev),
        _tensor(mass, "mass", torch.float32, side, dev), _tensor(pos, "pos", torch.int32, side, dev),
        _tensor(lens_out, "lens_out", torch.int32, (seqs,), dev),
        _tensor(mass_out, "mass_out", torch.float32, side, dev),
        _tensor(pos_out, "pos_out", torch.int32, side, dev), work.data_ptr(), N._nbytes(work),
        _status(status, dev), _stream(dev))
    _check(rc, "splitzip_kv4_evict")
    return lens_out, mass_out, pos_out
