"""A block-paged cache held in 4 bits: store, attention, rows read back.
Argument checks and marshalling only, as in paged.py, whose operators these
stand beside: block tables and slots are those of block_tables.

A pool is ``uint8 [num_blocks, Hk, block_size / 8, 9 d / 2]`` (make_pool_fp4): a
value is an e2m1 number times an e4m3 scale that 16 neighbours of a row share,
times a factor of the whole pool, 4.5 bits an element. Number times scale is
exact in bf16 and fp16. A step of the target:

  slots, kv_len, n_left = block_tables(ctx_len, out.kept_off, free, n_free, table, block_size, n_tokens=T)
  # for each layer, its pools and their factors:
  q = append_kv_fp4(k, v, slots, k_pool, v_pool, q=q, positions=out.kept_pos, cos_sin=cos_sin, n_new=out.n_kept)
  o = paged_attention_fp4(q, out.kept_off, kv_len, table, k_pool, v_pool, ws=ws)

Forward only: no gradient is recorded, and tensors are written without moving
their version counters.
"""

import ctypes

from . import _check, lib
from . import paged
from .paged import _handle, _new, torch_side


class _AppendShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_tokens", "n_q_heads", "n_kv_heads", "head_dim", "rotary_dim",
                                               "max_pos", "dtype", "block_size")]
                + [(n, ctypes.c_int64) for n in (
                    "pool_blocks", "q_stride_token", "q_stride_head", "qo_stride_token", "qo_stride_head",
                    "k_stride_token", "k_stride_head", "v_stride_token", "v_stride_head", "kp_stride_block",
                    "kp_stride_head", "vp_stride_block", "vp_stride_head")]
                + [("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)])


class _UnpackShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_kv_heads", "head_dim", "block_size", "dtype")]
                + [(n, ctypes.c_int64) for n in ("pool_blocks", "stride_block", "stride_head", "n_rows",
                                                 "o_stride_token", "o_stride_head")]
                + [("scale", ctypes.c_float), ("reserved", ctypes.c_int32)])


class _Shape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_seqs", "n_q_heads", "n_kv_heads", "head_dim", "dtype",
                                               "block_size", "table_stride", "n_tokens", "max_new", "reserved")]
                + [(n, ctypes.c_int64) for n in (
                    "dense_tokens", "pool_blocks", "q_stride_token", "q_stride_head", "o_stride_token",
                    "o_stride_head", "k_stride_block", "k_stride_head", "v_stride_block", "v_stride_head")])


class _Params(ctypes.Structure):
    _fields_ = [("causal", ctypes.c_int32), ("window", ctypes.c_int32), ("scale", ctypes.c_float),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float), ("spin_limit", ctypes.c_int32)]


def _bind(lib_):
    P, SZ, ref = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER
    sigs = {
        "sp_append_kv_fp4": [ref(_AppendShape)] + [P] * 12,
        "sp_unpack_fp4": [ref(_UnpackShape)] + [P] * 5,
        "sp_paged_attention_fp4_workspace": [ref(_Shape), ref(SZ)],
        "sp_paged_attention_fp4": [ref(_Shape), ref(_Params)] + [P] * 9 + [SZ, P],
    }
    for name, args in sigs.items():
        fn = getattr(lib_, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


def make_pool_fp4(num_blocks: int, block_size: int, n_kv_heads: int, head_dim: int, device="cuda"):
    """A zeroed 4-bit pool of keys or of values (block_size a multiple of 8,
    head_dim 64, 128 or 256)."""
    import torch
    if head_dim not in (64, 128, 256) or block_size < 8 or block_size % 8:
        raise ValueError("head_dim must be 64, 128 or 256 and block_size a multiple of 8")
    return torch.zeros(num_blocks, n_kv_heads, block_size // 8, 9 * head_dim // 2, dtype=torch.uint8, device=device)


def append_kv_fp4(k, v, slot_map, k_pool, v_pool, q=None, q_out=None, positions=None, cos_sin=None, n_new=None,
                  k_scale: float = 1.0, v_scale: float = 1.0, status=None, stream=None):
    """append_kv into 4-bit pools: keys (rotated in 32 bits) and values are
    stored without the pools' factors (from 2^-60 to 2^60); queries as there. The
    largest of 16 neighbours is stored as 6 times their scale, which reaches from
    2^-9 to 448: factors that bring it to between 0.1 and 2,688 keep all of the
    scale's bits. A group with an infinity or NaN reads back as NaN."""
    if q is not None and q_out is None:
        q_out = _new(q.shape, q.dtype, q, stream)
    rc = (paged._side or torch_side()).append_kv_fp4(k, v, slot_map, k_pool, v_pool, q, q_out, positions, cos_sin,
                                                     n_new, status, k_scale, v_scale, _handle(stream))
    if rc:
        _check(rc, "sp_append_kv_fp4")
    return q_out


def unpack_fp4(pool, dtype=None, slots=None, scale: float = 1.0, out=None, status=None, stream=None):
    """Rows of a 4-bit pool as bf16 (or fp16) values: all of them, [num_blocks,
    block_size, Hk, d] as specprefill_score_kv and paged_attention take a pool, or
    those at ``slots`` (int32, device; -1 gives zeros), [T, Hk, d]. ``scale`` is
    the pool's factor."""
    side = paged._side or torch_side()
    if out is None and stream is None:
        out = side.new_unpack_fp4(pool, slots, _is_half(dtype), scale, status)
        if isinstance(out, int):
            _check(out, "sp_unpack_fp4")
        return out
    if out is None:
        if pool.dim() != 4:
            raise ValueError("pool must be a 4-bit pool (make_pool_fp4)")
        blocks, hk, groups, width = pool.shape
        shape = (blocks, groups * 8, hk, width * 2 // 9) if slots is None else (slots.numel(), hk, width * 2 // 9)
        import torch
        out = _new(shape, torch.float16 if _is_half(dtype) else torch.bfloat16, pool, stream)
    rc = side.unpack_fp4(pool, slots, out, scale, status, _handle(stream))
    if rc:
        _check(rc, "sp_unpack_fp4")
    return out


_HALF = {"None": False, "torch.bfloat16": False, "torch.float16": True}


def _is_half(dtype):
    try:
        return _HALF[str(dtype)]
    except KeyError:
        raise ValueError("dtype must be bfloat16 or float16") from None


def _dense(kv_tokens, k_pool):
    return k_pool.shape[0] * k_pool.shape[2] * 8 if kv_tokens is None else int(kv_tokens)


class _Workspace:
    """Device workspace of paged_attention_fp4 and what it was made for."""

    def __init__(self, buffer, dense):
        self.buffer = buffer
        self.dense = dense

    def data_ptr(self):
        return self.buffer.data_ptr()

    def numel(self):
        return self.buffer.numel()


def make_attention_fp4_workspace(q, n_seqs: int, k_pool, max_new=None, kv_tokens=None, stream=None):
    """Workspace of paged_attention_fp4 for queries of q's shape (its rows bound
    the new tokens of a call) of ``n_seqs`` requests over pools like ``k_pool``;
    calls that share one must be ordered. Requests with many new tokens are
    computed over a 16-bit copy of their cached tokens in the workspace:
    ``kv_tokens`` bounds those tokens (default: as many as the pool has, so that the
    workspace is 3.6 times as large as both pools of a layer; one serves all layers).
    Requests that do not fit are computed from the 4-bit rows, a long chunk several times
    more slowly, and so is every one behind the first of them. With a small
    ``max_new``, the most new tokens of a request, none is needed."""
    import torch
    dense = _dense(kv_tokens, k_pool)
    n = torch_side().workspace_fp4(q, n_seqs, k_pool, max_new, dense)
    if n < 0:
        _check(-n, "sp_paged_attention_fp4_workspace")
    ws = _new(n + 256, torch.uint8, q, stream)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n]
    handle = torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream
    _check(lib().sp_workspace_init(ws.data_ptr(), n, handle), "sp_workspace_init")
    return _Workspace(ws, dense)


def paged_attention_fp4(q, q_off, kv_len, block_table, k_pool, v_pool, causal: bool = True, window: int = 0,
                        scale: float = 0.0, k_scale: float = 1.0, v_scale: float = 1.0, out=None, lse=None,
                        max_new=None, ws=None, stream=None, spin_limit: int = 0):
    """paged_attention over 4-bit pools with the factors ``k_scale`` and
    ``v_scale``: the attention over the values that unpack_fp4 gives, with
    the same arguments, masks and outputs. ``max_new`` (default: the rows of q) is the most
    new tokens of a request; a decode step that says 1 launches less. ``ws`` from
    make_attention_fp4_workspace, with its status in device_status; without
    it the call allocates one (of the default size), whose status is lost."""
    if out is None:
        out = _new(q.shape, q.dtype, q, stream)
    if q.shape[0] == 0:
        return out
    if ws is None:
        ws = make_attention_fp4_workspace(q, kv_len.numel(), k_pool, max_new, None, stream)
    rc = (paged._side or torch_side()).paged_attention_fp4(
        q, q_off, kv_len, block_table, k_pool, v_pool, causal, window, scale, k_scale, v_scale, out, lse, max_new,
        ws.buffer, ws.dense, spin_limit, _handle(stream))
    if rc:
        _check(rc, "sp_paged_attention_fp4")
    return out
