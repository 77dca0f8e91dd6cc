"""Sparse prefill on a block-paged cache: block tables and slots of a step,
rotation and store of its new tokens, attention over the cache. Argument
checks and marshalling only, like the rest of the binding; the checks and the
calls of the C ABI are in a small extension over torch's tensors
(csrc/sp_paged_torch.cpp), since a decode step makes them for every layer. The
ctypes structs below mirror the ABI for callers without torch.

A cache layer is two pools ``[num_blocks, block_size, Hk, d]`` (bf16 or fp16,
d contiguous, rows evenly strided), as ``kv_source`` takes them; block tables
are int32 ``[B, max_blocks]``. A step of the target, with no host round trip
after the scoring call that gave ``out``:

  slots, kv_len, n_left = block_tables(ctx_len, out.kept_off, free, n_free, table, block_size, n_tokens=T)
  # for each layer:
  q = append_kv(k, v, slots, k_pool, v_pool, q=q, positions=out.kept_pos, cos_sin=cos_sin, n_new=out.n_kept)
  o = paged_attention(q, out.kept_off, kv_len, table, k_pool, v_pool, ws=ws)

Forward only: no gradient is recorded, and tensors are written without moving
their version counters.
"""

import ctypes
import importlib.machinery
import importlib.util
import os

from . import LIB_PATH, _build, _check, lib


class _BlockShape(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("table_stride", ctypes.c_int32), ("n_tokens", ctypes.c_int32),
                ("free_capacity", ctypes.c_int32), ("pool_blocks", ctypes.c_int32)]


class _AppendShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_tokens", "n_q_heads", "n_kv_heads", "head_dim", "rotary_dim",
                                               "max_pos", "dtype", "reserved")]
                + [(n, ctypes.c_int64) for n in (
                    "pool_tokens", "q_stride_token", "q_stride_head", "qo_stride_token", "qo_stride_head",
                    "k_stride_token", "k_stride_head", "v_stride_token", "v_stride_head", "kp_stride_token",
                    "kp_stride_head", "vp_stride_token", "vp_stride_head")])


class _PagedShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_seqs", "n_q_heads", "n_kv_heads", "head_dim", "dtype",
                                               "block_size", "table_stride", "n_tokens")]
                + [(n, ctypes.c_int64) for n in (
                    "pool_tokens", "q_stride_token", "q_stride_head", "o_stride_token", "o_stride_head",
                    "k_stride_token", "k_stride_head", "v_stride_token", "v_stride_head")])


class _AttnParams(ctypes.Structure):
    _fields_ = [("causal", ctypes.c_int32), ("window", ctypes.c_int32), ("scale", ctypes.c_float),
                ("spin_limit", ctypes.c_int32)]


def _bind(lib_):
    P, SZ, ref = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER
    sigs = {
        "sp_block_tables": [ref(_BlockShape)] + [P] * 10,
        "sp_append_kv": [ref(_AppendShape)] + [P] * 12,
        "sp_paged_attention_workspace": [ref(_PagedShape), ref(SZ)],
        "sp_paged_attention": [ref(_PagedShape), ref(_AttnParams)] + [P] * 9 + [SZ, P],
    }
    for name, args in sigs.items():
        fn = getattr(lib_, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


_side = None


def torch_side():
    """The extension, loaded once (raises if it is missing)."""
    global _side
    if _side is None:
        import torch  # noqa: F401  (its libraries are loaded before the extension that uses them)
        lib()
        path = os.path.join(os.path.dirname(LIB_PATH), "_paged_torch.so")
        if not _build.torch_side_fits():
            raise RuntimeError(f"_paged_torch.so not built for this torch and Python ({path}); "
                               "run __graft_entry__.build()")
        loader = importlib.machinery.ExtensionFileLoader("_paged_torch", path)
        spec = importlib.util.spec_from_file_location("_paged_torch", path, loader=loader)
        side = importlib.util.module_from_spec(spec)
        loader.exec_module(side)
        _side = side
    return _side


def _new(shape, dtype, like, stream):
    """An output or workspace that belongs to the call's stream."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def block_tables(ctx_len, new_off, free_blocks, n_free, block_table, block_size: int, n_tokens=None, slot_map=None,
                 kv_len=None, n_left=None, status=None, pool_blocks=None, stream=None):
    """(slot_map, kv_len, n_left) of a step, and its new blocks in
    ``block_table`` (int32 [B, max_blocks], in place). All int32 on the device:
    ``ctx_len`` [B] tokens cached before the step, ``new_off`` [B+1] offsets
    of its new tokens (the scoring call's kept_off), ``free_blocks`` with the
    ids [0, n_free) free (taken from the end), ``n_free`` [1]. ``slot_map``
    holds ``n_tokens`` entries (at least new_off[B]), -1 behind the last new
    token; ``n_left`` [1] counts the blocks that stay free. ``status`` [1],
    zeroed by the caller, is raised to a STATUS code when the free list is too
    short (SP_ERR_CAPACITY) or a length is out of range (SP_ERR_DEVICE): the
    call then takes nothing, every slot is -1 and every kv_len 0. Where steps
    are chained on the device, kv_len and n_left become ctx_len and n_free only
    where status is still 0: ``ctx_len.copy_(torch.where(status == 0, kv_len,
    ctx_len))``, and n_free alike. ``pool_blocks`` bounds the block ids."""
    if slot_map is None:
        if n_tokens is None:
            raise ValueError("give slot_map or n_tokens")
        slot_map = _new(int(n_tokens), ctx_len.dtype, ctx_len, stream)
    if kv_len is None:
        kv_len = _new(ctx_len.numel(), ctx_len.dtype, ctx_len, stream)
    if n_left is None:
        n_left = _new(1, ctx_len.dtype, ctx_len, stream)
    rc = (_side or torch_side()).block_tables(
        ctx_len, new_off, free_blocks, n_free, block_table, block_size, n_tokens, slot_map, kv_len, n_left, status,
        pool_blocks, _handle(stream))
    if rc:
        _check(rc, "sp_block_tables")
    return slot_map, kv_len, n_left


def append_kv(k, v, slot_map, k_pool, v_pool, q=None, q_out=None, positions=None, cos_sin=None, n_new=None,
              status=None, stream=None):
    """Store the new tokens' keys ``k`` and values ``v`` [T, Hk, d] (strided
    views are fine) in the pools at ``slot_map`` (int32, device; -1 stores
    nothing), keys rotated to ``positions`` (int32, device) when ``cos_sin``
    (fp32 [max_pos, rotary_dim]: cosines, then sines) is given; returns
    ``q_out`` [T, Hq, d], the rotated ``q`` (``q_out=q`` rotates in place), or
    None without queries. ``n_new`` (int32 [1], device) bounds the rows in
    use. Slots must differ from one another. ``status`` as in block_tables."""
    if q is not None and q_out is None:
        q_out = _new(q.shape, q.dtype, q, stream)
    rc = (_side or torch_side()).append_kv(k, v, slot_map, k_pool, v_pool, q, q_out, positions, cos_sin, n_new, status,
                                           _handle(stream))
    if rc:
        _check(rc, "sp_append_kv")
    return q_out


def make_attention_workspace(q, n_seqs: int, k_pool, stream=None):
    """Workspace of paged_attention for queries of q's shape (its rows bound
    the new tokens of a call) of ``n_seqs`` requests over pools like
    ``k_pool``; calls that share one must be ordered."""
    import torch
    n = torch_side().workspace(q, n_seqs, k_pool)
    if n < 0:
        _check(-n, "sp_paged_attention_workspace")
    ws = _new(n + 256, torch.uint8, q, stream)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n]
    handle = torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream
    _check(lib().sp_workspace_init(ws.data_ptr(), n, handle), "sp_workspace_init")
    return ws


def paged_attention(q, q_off, kv_len, block_table, k_pool, v_pool, causal: bool = True, window: int = 0,
                    scale: float = 0.0, out=None, lse=None, ws=None, stream=None, spin_limit: int = 0):
    """Attention of the new tokens ``q`` [T, Hq, d] over the paged cache:
    request b's are rows [q_off[b], q_off[b+1]), the last of its ``kv_len[b]``
    cached tokens (int32, device). Each sees the cached tokens up to itself
    (``causal``), only the last ``window`` of them when window > 0, or all.
    Returns ``out`` (like q; rows behind q_off[B] are not written); ``lse``
    (fp32 [T, Hq], optional) receives the log-sum-exp of the scaled logits.
    A row that sees nothing gives 0 and -inf. ``ws`` from
    make_attention_workspace, with its status in device_status; without it
    the call allocates one (20 to 40 MB), whose status is lost."""
    if out is None:
        out = _new(q.shape, q.dtype, q, stream)
    if q.shape[0] == 0:
        return out
    if ws is None:
        ws = make_attention_workspace(q, kv_len.numel(), k_pool, stream)
    rc = (_side or torch_side()).paged_attention(q, q_off, kv_len, block_table, k_pool, v_pool, causal, window, scale,
                                                 out, lse, ws, spin_limit, _handle(stream))
    if rc:
        _check(rc, "sp_paged_attention")
    return out
