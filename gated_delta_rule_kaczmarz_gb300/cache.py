"""Binding of the paged key/value cache in 4 bits: rows appended and read back,
attention over it, and the pages' operators (fork, free, growth, trimming,
compaction, copies).

The same rules as in ``attention``: argument marshalling only, a non-OK status
raises ``KlaError``, and a call runs on the device of its tensors.  A cache is a
pool of pages, uint8 [n_pages, Hk, page / 16, 18 d] (``kla_kv4_pool``), and its
book: table int32 [B, columns] of page numbers, lens int32 [B], refs int32
[n_pages] with the number of sequences that hold each page.  A step of a decode
loop: ``kla_pages_grow`` makes room, ``kla_kv4_append`` writes the new rows,
``kla_kv4_attn`` attends over them, and ``kla_pages_trim`` takes back the positions of
drafted tokens that are not taken.
"""
from __future__ import annotations

import functools
import math
from operator import attrgetter, index

import torch

from .attention import _dense, _given, _refuse, _rows, _scale, _type_code
from .binding import KlaError, load

_INT = torch.int32


@functools.lru_cache(maxsize=1024)
def _size(device, name, args):
    """A workspace's size, asked for once: it goes by the device and the sizes alone."""
    with torch.cuda.device(device):
        return getattr(load(), name)(*args)


def _of_torch(name):
    """A function of torch's own library that a small call is faster with; None where this torch
    has none of that name, and torch.empty takes its place."""
    try:
        return attrgetter(name)(torch._C)
    except AttributeError:
        return None


#: What compiled graphs take their buffers with, on the current device: 1.5 us of a small call
#: where torch.empty takes 4.
_empty = _of_torch("_dynamo.guards._empty_strided_cuda")
#: torch's allocator without a tensor around it: 0.7 us a call, not 5.
_alloc = _of_torch("_cuda_cudaCachingAllocator_raw_alloc")
_free = _of_torch("_cuda_cudaCachingAllocator_raw_delete")


@functools.lru_cache(maxsize=1024)
def _steps(size):
    """The strides of a dense tensor."""
    return tuple(math.prod(size[i + 1:]) for i in range(len(size)))


def _out(t, name, size, dtype, dev):
    """A dense output, made where there is none, and its address; size: a tuple."""
    if t is None:
        if _empty is not None and torch._C._cuda_getDevice() == dev:
            t = _empty(size, _steps(size), dtype)
        else:
            t = torch.empty(size, dtype=dtype, device=dev)
        return t, t.data_ptr()
    return t, _dense(t, name, dtype, dev, size)


def _run(fn, dev, args, name, sizes, workspace, check):
    """Runs a library call with its workspace, of the size that name(*sizes) says (name None:
    none), and the stream last in the arguments."""
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _run(fn, dev, args, name, sizes, workspace, check)
    need, own = 0 if name is None else _size(dev, name, sizes), None
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if workspace is not None:
        at, have = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        if workspace.get_device() != dev:
            raise ValueError(f"workspace must be on cuda:{dev}, got {workspace.device}")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if have < need:
            raise ValueError(f"workspace needs {need} bytes")
        need = have
    elif not need:
        at = None
    elif _alloc is None or _free is None:
        kept = torch.empty(need, dtype=torch.uint8, device=dev)     # until the call is enqueued
        at = kept.data_ptr()
    else:
        # given back once the call is enqueued, for what comes behind it in the stream
        at = own = _alloc(need, stream)
    try:
        status = fn(*args, at, need, stream)
        if check and not status:
            status = load().kla_workspace_status(at, need, stream)
    finally:
        if own is not None:
            _free(own)
    if status:
        lib = load()
        raise KlaError(status, lib.kla_last_error_message().decode() or
                       lib.kla_status_str(status).decode())


def kla_kv4_page_bytes(page, Hk, d) -> int:
    return int(load().kla_kv4_page_bytes(page, Hk, d))


def kla_kv4_attn_workspace_size(B, Tq, Hq, Hk, d, page, columns, dtype=1) -> int:
    return int(load().kla_kv4_attn_workspace_size(B, Tq, Hq, Hk, d, page, columns, dtype))


def kla_pages_workspace_size(S, columns, n_pages, n=0) -> int:
    return int(load().kla_pages_workspace_size(S, columns, n_pages, n))


def kla_kv4_pool(n_pages, page, Hk, d, layers=None, device="cuda"):
    """An empty pool: uint8 [n_pages, Hk, page / 16, 18 d], with `layers` one of
    them for each layer ([layers, ...]: pool[i] for a layer's calls, the whole for
    kla_pages_*)."""
    if not kla_kv4_page_bytes(page, Hk, d):
        raise ValueError("page must be a multiple of 16 and d 64 or 128 "
                         f"(got page={page} Hk={Hk} d={d})")
    shape = (n_pages, Hk, page // 16, 18 * d)
    return torch.zeros(shape if layers is None else (layers, *shape), dtype=torch.uint8,
                       device=device)


# A small call takes about as long as its checks do, so these look over in one go what is
# nearly always right; what is not is looked at again, to say what is wrong.
def _book(table, lens, dev):
    """The addresses of table and lens."""
    size = table.shape
    if (len(size) == 2 and dev >= 0 and table.get_device() == dev and lens.get_device() == dev
            and table.dtype is _INT and lens.dtype is _INT and lens.shape == (size[0],)
            and table.is_contiguous() and lens.is_contiguous()):
        return table.data_ptr(), lens.data_ptr()
    if dev < 0:
        raise ValueError("table must be a CUDA tensor")
    if len(size) != 2:
        raise ValueError(f"table must have shape [B, columns], got {tuple(size)}")
    return _dense(table, "table", _INT, dev, size), _dense(lens, "lens", _INT, dev, size[:1])


def _pool(pool, dev, Hk=None, d=None):
    """The address of a layer's pool, Hk, d, a page's tokens and the pages."""
    shape = pool.shape
    if len(shape) != 4:
        raise ValueError("pool must have shape [n_pages, Hk, page / 16, 18 d], got "
                         f"{tuple(shape)}")
    n_pages, heads, blocks, size = shape
    d = size // 18 if d is None else d
    if (size != 18 * d or pool.dtype is not torch.uint8 or pool.get_device() != dev or dev < 0
            or (Hk is not None and heads != Hk)):
        _refuse(pool, "pool", torch.uint8, dev, (n_pages, heads if Hk is None else Hk, blocks, 18 * d))
    if not pool.is_contiguous():
        raise ValueError("pool must be contiguous")
    return pool.data_ptr(), heads, d, 16 * blocks, n_pages


def _rows_call(fn, k, v, pool, table, lens, cu_seqlens, k_unit, v_unit, workspace, check):
    kind, dev, shape, cu = k.dtype, pool.get_device(), k.shape, None
    packed = cu_seqlens is not None
    if len(shape) != (3 if packed else 4):
        raise ValueError(f"k must have shape {'[total, Hk, d]' if packed else '[B, T, Hk, d]'}, "
                         f"got {tuple(shape)}")
    T, hk, d = shape[-3:]
    dt = _type_code(k)
    at, hk, d, page, n_pages = _pool(pool, dev, hk, d)
    rows, lengths = _book(table, lens, dev)
    B, columns = table.shape
    if packed:
        cu = _dense(cu_seqlens, "cu_seqlens", _INT, dev, (B + 1,))
    elif shape[0] != B:
        shape = (B, T, hk, d)
    if (v.dtype is kind and k.get_device() == dev and v.get_device() == dev and k.shape == shape
            and v.shape == shape and k.is_contiguous() and v.is_contiguous()):
        ks = vs = hk * d
    else:
        ks, vs = _rows(k, "k", kind, dev, shape), _rows(v, "v", kind, dev, shape)
    if check and workspace is None:
        workspace = torch.empty(256, dtype=torch.uint8, device=pool.device)
    _run(fn, dev, (k.data_ptr(), ks, v.data_ptr(), vs, at, rows, lengths, cu, k_unit, v_unit, B, T,
                   hk, d, page, n_pages, columns, dt), None, None, workspace, check)


def kla_kv4_append(k, v, pool, table, lens, cu_seqlens=None, k_unit=1.0, v_unit=1.0,
                   workspace=None, stream=None, check_status=False):
    """Writes rows of keys and values to the places of each sequence's last
    positions (lens counts them already).  k, v: [B,T,Hk,d], or packed [total,Hk,d]
    with cu_seqlens int32 [B+1]; views of a fused projection's output among them.
    Rows before position 0 and behind the table's last column are left out.  k_unit,
    v_unit: powers of two, the same in every call on a cache.  check_status waits for
    the call and raises what the device reports."""
    if stream is not None:
        with _given(stream, pool):
            return kla_kv4_append(k, v, pool, table, lens, cu_seqlens, k_unit, v_unit, workspace,
                                  check_status=check_status)
    _rows_call(load().kla_kv4_append, k, v, pool, table, lens, cu_seqlens, k_unit, v_unit,
               workspace, check_status)


def kla_kv4_read(pool, table, lens, T=None, total=None, cu_seqlens=None, dtype=torch.bfloat16,
                 k_unit=1.0, v_unit=1.0, k_out=None, v_out=None, workspace=None, stream=None,
                 check_status=False):
    """The inverse of kla_kv4_append: the last T positions of each sequence,
    [B,T,Hk,d], or packed rows [total,Hk,d] with cu_seqlens; rows before position 0
    are zeros.  k_out, v_out: written where given, views among them.  Returns
    (k, v)."""
    if stream is not None:
        with _given(stream, pool):
            return kla_kv4_read(pool, table, lens, T, total, cu_seqlens, dtype, k_unit, v_unit,
                                k_out, v_out, workspace, check_status=check_status)
    if (T is None) == (cu_seqlens is None) or (total is None) != (cu_seqlens is None):
        raise ValueError("T must be given, or total and cu_seqlens")
    if pool.dim() != 4:
        _pool(pool, pool.get_device())
    hk, d, dev = pool.shape[1], pool.shape[3] // 18, pool.get_device()
    if dev < 0:
        raise ValueError("pool must be a CUDA tensor")
    n = index(T if cu_seqlens is None else total)
    if n < 0:
        raise ValueError(f"{'T' if cu_seqlens is None else 'total'} must not be negative, got {n}")
    shape = (table.shape[0], n, hk, d) if cu_seqlens is None else (n, hk, d)
    if k_out is None:
        k_out = _out(None, "k_out", shape, dtype, dev)[0]
    elif k_out.shape != shape:
        _refuse(k_out, "k_out", dtype, dev, shape)
    if v_out is None:
        v_out = _out(None, "v_out", shape, k_out.dtype, dev)[0]
    _rows_call(load().kla_kv4_read, k_out, v_out, pool, table, lens, cu_seqlens, k_unit, v_unit,
               workspace, check_status)
    return k_out, v_out


def kla_kv4_attn(q, pool, table, lens, scale=None, k_unit=1.0, v_unit=1.0, o=None, lse=None,
                 return_lse=True, workspace=None, stream=None, check_status=False):
    """Causal attention with grouped heads over a paged 4-bit cache.  q:
    [B,Tq,Hq,d], the last Tq positions of each sequence; query i sees the positions
    j <= i + lens - Tq; scale: 1/sqrt(d) unless given.  Returns (o, lse), o dense,
    lse [B,Tq,Hq] fp32 (None with return_lse=False).  Many query rows in bf16 (128 to a
    key head and more) take up to 1 GiB of workspace, by the table's width."""
    if stream is not None:
        with _given(stream, q):
            return kla_kv4_attn(q, pool, table, lens, scale, k_unit, v_unit, o, lse, return_lse,
                                workspace, check_status=check_status)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError(f"q must have shape [B, Tq, Hq, d], got {tuple(shape)}")
    dt, dev, kind = _type_code(q), q.get_device(), q.dtype
    B, Tq, hq, d = shape
    qs = hq * d if q.is_contiguous() and dev >= 0 else _rows(q, "q", kind, dev, shape)
    at, hk, d, page, n_pages = _pool(pool, dev, None, d)
    rows, lengths = _book(table, lens, dev)
    if table.shape[0] != B:
        raise ValueError(f"table must have {B} rows, got {tuple(table.shape)}")
    columns = table.shape[1]
    o, out = _out(o, "o", (B, Tq, hq, d), kind, dev)
    stats = None
    if return_lse or lse is not None:
        lse, stats = _out(lse, "lse", (B, Tq, hq), torch.float32, dev)
    _run(load().kla_kv4_attn, dev,
         (q.data_ptr(), qs, at, rows, lengths, _scale(scale, d), k_unit, v_unit, out, stats, B, Tq,
          hq, hk, d, page, n_pages, columns, dt),
         "kla_kv4_attn_workspace_size", (B, Tq, hq, hk, d, page, columns, dt), workspace,
         check_status)
    return o, lse


# ---------------------------------------------------------------------- pages
def _layers(pool, n_pages):
    """The address of all layers' pages, their number and a page's bytes."""
    if pool.dim() < 2 or (n_pages is not None and pool.shape[1] != n_pages):
        raise ValueError(f"pool must have shape [layers, {n_pages or 'n_pages'}, ...], got "
                         f"{tuple(pool.shape)}")
    if not pool.is_contiguous():
        raise ValueError("pool must be contiguous")
    layers, n = pool.shape[:2]
    return pool.data_ptr(), layers, pool.numel() // max(1, layers * n) * pool.element_size()


def _held(table, lens, refs):
    """The device, the pages' number, the sizes of the table and the book's addresses."""
    dev, n_pages = table.get_device(), refs.numel()
    return dev, n_pages, table.shape, (*_book(table, lens, dev),
                                       _dense(refs, "refs", _INT, dev, (n_pages,)))


_PAGES = "kla_pages_workspace_size"      # of (S, columns, n_pages, n)


def kla_pages_fork(table, lens, refs, src, dst, page, workspace=None, stream=None,
                   check_status=False):
    """Sequence dst[f] becomes what src[f] was before the call, for all f at once:
    its length and its pages, shared (src[f] = -1: empty).  src, dst: int32 [n] on
    the device, dst without repetition.  Changes table, lens and refs."""
    if stream is not None:
        with _given(stream, table):
            return kla_pages_fork(table, lens, refs, src, dst, page, workspace,
                                  check_status=check_status)
    dev, n_pages, (S, columns), book = _held(table, lens, refs)
    n = dst.numel()
    to = _dense(dst, "dst", _INT, dev, (n,))
    of = _dense(src, "src", _INT, dev, (n,))
    _run(load().kla_pages_fork, dev, (*book, of, to, S, columns, page, n_pages, n), _PAGES,
         (S, columns, n_pages, n), workspace, check_status)


def kla_pages_free(table, lens, refs, seqs, page, workspace=None, stream=None,
                   check_status=False):
    """The sequences seqs (int32 [n]) become empty; pages that nobody holds any
    more are free."""
    kla_pages_fork(table, lens, refs, None, seqs, page, workspace, stream, check_status)


def kla_pages_grow(pool, table, lens, refs, n_new, page, workspace=None, stream=None,
                   check_status=False):
    """Room for n_new[s] (int32 [S]) more positions of every sequence; lens counts
    them.  A shared last page that is partly filled is copied first, in all layers of
    the pool ([layers, n_pages, ...], any type).  check_status raises
    KLA_ERR_PAGES where there are not enough free pages; nothing has changed then."""
    if stream is not None:
        with _given(stream, table):
            return kla_pages_grow(pool, table, lens, refs, n_new, page, workspace,
                                  check_status=check_status)
    dev, n_pages, (S, columns), book = _held(table, lens, refs)
    more = _dense(n_new, "n_new", _INT, dev, (S,))
    if pool.get_device() != dev:
        _refuse(pool, "pool", pool.dtype, dev, pool.shape)
    _run(load().kla_pages_grow, dev,
         (*_layers(pool, n_pages), *book, more, S, columns, page, n_pages), _PAGES,
         (S, columns, n_pages, 0), workspace, check_status)


def kla_pages_trim(table, lens, refs, n_cut, page, workspace=None, stream=None,
                   check_status=False):
    """The last n_cut[s] (int32 [S]) positions of every sequence are given up, drafted
    tokens that were not taken; pages that nobody holds any more are free."""
    if stream is not None:
        with _given(stream, table):
            return kla_pages_trim(table, lens, refs, n_cut, page, workspace,
                                  check_status=check_status)
    dev, n_pages, (S, columns), book = _held(table, lens, refs)
    cut = _dense(n_cut, "n_cut", _INT, dev, (S,))
    _run(load().kla_pages_trim, dev, (*book, cut, S, columns, page, n_pages), _PAGES,
         (S, columns, n_pages, 0), workspace, check_status)


def kla_pages_compact(pool, table, lens, refs, page, page_map=None, n_used=None, workspace=None,
                      stream=None, check_status=False):
    """Pages in use move below n_used, the number of them, in all layers of the
    pool.  Returns (page_map, n_used): int32 [n_pages], where each page is now (-1:
    free), and int32 [1], on the device."""
    if stream is not None:
        with _given(stream, table):
            return kla_pages_compact(pool, table, lens, refs, page, page_map, n_used, workspace,
                                     check_status=check_status)
    dev, n_pages, (S, columns), book = _held(table, lens, refs)
    page_map, where = _out(page_map, "page_map", (n_pages,), _INT, dev)
    n_used, count = _out(n_used, "n_used", (1,), _INT, dev)
    if pool.get_device() != dev:
        _refuse(pool, "pool", pool.dtype, dev, pool.shape)
    _run(load().kla_pages_compact, dev,
         (*_layers(pool, n_pages), *book, where, count, S, columns, page, n_pages), _PAGES,
         (S, columns, n_pages, 0), workspace, check_status)
    return page_map, n_used


def kla_pages_copy(pool, src, dst, workspace=None, stream=None, check_status=False):
    """The contents of pages src[i] to dst[i] in all layers of the pool ([layers,
    n_pages, ...], any type; KLA's states [B,H,dk,dv] as S[None]).  No target may be
    there twice or be the source of another."""
    if stream is not None:
        with _given(stream, pool):
            return kla_pages_copy(pool, src, dst, workspace, check_status=check_status)
    dev, n = pool.get_device(), dst.numel()
    if dev < 0:
        raise ValueError("pool must be a CUDA tensor")
    at, layers, size = _layers(pool, None)
    n_pages = pool.shape[1]
    of, to = _dense(src, "src", _INT, dev, (n,)), _dense(dst, "dst", _INT, dev, (n,))
    _run(load().kla_pages_copy, dev, (at, layers, size, of, to, n_pages, n), _PAGES,
         (0, 0, n_pages, n), workspace, check_status)
