"""Pages of the block-paged caches (16-bit or 4-bit): requests forked, cut and
freed, rows and blocks copied. Argument checks and marshalling only, as in
paged.py; block tables, free lists and lengths are those of block_tables.

``shared`` (int32 [num_blocks], zeros at first) counts a block's holders beyond
the first. Several continuations of one prompt:

  kv_len, copy_src, copy_dst, n_left = fork_blocks(src, dst, ctx_len, table, shared, free, n_free, block_size)
  copy_kv(pools, copy_src, copy_dst, rows=block_size)       # the begun blocks, in all layers at once
  ...                                                       # steps of the forks; later, where new_len is 0:
  kv_len, n_left = free_blocks(ctx_len, new_len, table, shared, free, n_free, block_size)

A request whose cut ends inside a shared block goes on in another row (``row``, empty before):

  kv_len, n_left = free_blocks(ctx_len, new_len, table, shared, free, n_free, block_size)
  kv_len, copy_src, copy_dst, n_left = fork_blocks(cut, row, kv_len, table, shared, free, n_left, block_size)
  copy_kv(pools, copy_src, copy_dst, rows=block_size)
  kv_len, n_left = free_blocks(kv_len, without_cut, table, shared, free, n_left, block_size)

The kept tokens of a cached prompt moved to blocks of their own (``new_table``
has a row for each prompt, empty before):

  slots, kv_len, n_left = block_tables(zeros, out.kept_off, free, n_free, new_table, block_size, n_tokens=T)
  copy_kv(pools, out.kept_pos, slots, block_table=table, src_off=out.kept_off, n=out.n_kept)
"""

import ctypes

from . import _check
from . import paged
from .paged import _handle, _new, torch_side


class _CopyShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_pools", "n_entries", "rows", "block_size", "n_kv_heads",
                                               "head_dim", "fp4", "n_seqs", "table_stride", "reserved")]
                + [(n, ctypes.c_int64) for n in ("pool_blocks", "stride_block", "stride_token", "stride_head")])


class _PagesShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_seqs", "n_forks", "block_size", "table_stride", "pool_blocks",
                                              "free_capacity", "alone")]


def _bind(lib_):
    P, ref = ctypes.c_void_p, ctypes.POINTER
    sigs = {
        "sp_copy_kv": [ref(_CopyShape), ref(P)] + [P] * 7,
        "sp_fork_blocks": [ref(_PagesShape)] + [P] * 13,
        "sp_free_blocks": [ref(_PagesShape)] + [P] * 10,
    }
    for name, args in sigs.items():
        fn = getattr(lib_, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


def copy_kv(pools, src, dst, rows: int = 1, block_table=None, src_off=None, n=None, status=None, stream=None):
    """Copies rows of the cache in every one of ``pools`` (a sequence of at most
    256 pools of one shape). Entry i copies the ``rows`` consecutive slots from
    src[i] * rows on to those from dst[i] * rows on (int32, device; -1: nothing):
    single tokens, or with rows=block_size whole blocks. With ``block_table`` and
    ``src_off`` (int32 [B+1]), src[i] is a cached token of the request b with
    src_off[b] <= i < src_off[b+1]. ``n`` (int32 [1], device) bounds the entries in use.
    Slots written differ from one another and from all slots read. ``status`` as
    in block_tables."""
    rc = (paged._side or torch_side()).copy_kv(pools, src, dst, rows, block_table, src_off, n, status, _handle(stream))
    if rc:
        _check(rc, "sp_copy_kv")


def fork_blocks(src, dst, ctx_len, block_table, shared, free_blocks, n_free, block_size: int, kv_len=None,
                copy_src=None, copy_dst=None, n_left=None, status=None, stream=None):
    """(kv_len, copy_src, copy_dst, n_left): row dst[i] of ``block_table`` becomes
    a request with the cached tokens of row src[i] (int32, device; src -1: no
    fork). Full blocks are shared, a begun last one is taken from the free list's
    end and named in copy_src and copy_dst (block ids, -1: nothing) for copy_kv
    with rows=block_size. Rows dst hold nothing before (ctx_len 0), differ from one
    another and are in no src. ``status`` as in block_tables: a call that fails
    forks nothing, and its kv_len is ctx_len."""
    if kv_len is None:
        kv_len = _new(ctx_len.numel(), ctx_len.dtype, ctx_len, stream)
    if copy_src is None:
        copy_src = _new(src.numel(), ctx_len.dtype, ctx_len, stream)
    if copy_dst is None:
        copy_dst = _new(src.numel(), ctx_len.dtype, ctx_len, stream)
    if n_left is None:
        n_left = _new(1, ctx_len.dtype, ctx_len, stream)
    rc = (paged._side or torch_side()).fork_blocks(src, dst, ctx_len, block_table, shared, free_blocks, n_free,
                                                   block_size, kv_len, copy_src, copy_dst, n_left, status,
                                                   _handle(stream))
    if rc:
        _check(rc, "sp_fork_blocks")
    return kv_len, copy_src, copy_dst, n_left


def free_blocks(ctx_len, new_len, block_table, shared, free_blocks, n_free, block_size: int, kv_len=None, n_left=None,
                status=None, stream=None, alone: bool = False):
    """(kv_len, n_left): every request cut from ctx_len[b] to new_len[b] cached
    tokens (0: it ends). Blocks that nobody holds any more go behind the n_free
    free ones in ``free_blocks`` (in place), in the order of their ids; ``n_left``
    counts the free ones afterwards. ``status`` as in block_tables: a call that
    fails (a block let go more often than held, a full list) frees nothing,
    and its kv_len is ctx_len.

    A request cut inside a block that others hold as well may be read, but not
    filled further: its next tokens would overwrite theirs. To go on with it, fork it
    into an empty row, which gets the begun block as a copy of its own, and free the
    row that was cut. ``alone=True`` refuses such cuts (status as for a bad length)."""
    if kv_len is None:
        kv_len = _new(ctx_len.numel(), ctx_len.dtype, ctx_len, stream)
    if n_left is None:
        n_left = _new(1, ctx_len.dtype, ctx_len, stream)
    rc = (paged._side or torch_side()).free_blocks(ctx_len, new_len, block_table, shared, free_blocks, n_free,
                                                   block_size, kv_len, n_left, status, alone, _handle(stream))
    if rc:
        _check(rc, "sp_free_blocks")
    return kv_len, n_left
