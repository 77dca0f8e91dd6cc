"""Sparse prefill on a block-paged cache: block tables and slots of a step,
rotation and store of its new tokens, attention over the cache. Argument
checks and marshalling only, like the rest of the binding.

A cache layer is two pools ``[num_blocks, block_size, Hk, d]`` (bf16 or fp16,
d contiguous, rows evenly strided), as ``kv_source`` takes them; block tables
are int32 ``[B, max_blocks]``. A step of the target, with no host round trip
after the scoring call that gave ``out``:

  slots, kv_len, n_left = block_tables(ctx_len, out.kept_off, free, n_free, table, block_size, n_tokens=T)
  # for each layer:
  q = append_kv(k, v, slots, k_pool, v_pool, q=q, positions=out.kept_pos, cos_sin=cos_sin, n_new=out.n_kept)
  o = paged_attention(q, out.kept_off, kv_len, table, k_pool, v_pool, ws=ws)
"""

import ctypes

from . import _SZ, _check, lib


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


_INT32_MAX = 2 ** 31 - 1
_int32 = _float32 = _codes = _raw_stream = _current_device = None


def _init():
    """torch's types and stream lookup, looked up once: a decode step makes
    these calls for every layer, and the host's part of them is most of it
    (torch.cuda.current_stream() alone takes 3 us, the raw handle 0.1)."""
    global _int32, _float32, _codes, _raw_stream, _current_device
    import torch
    _int32, _float32 = torch.int32, torch.float32
    _codes = {torch.bfloat16: 0, torch.float16: 1}
    _current_device = torch.cuda.current_device
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)


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


def _device_of(t, name) -> int:
    """The device of a call: that of its first tensor, which has to be the
    current CUDA device (the library launches there)."""
    if _int32 is None:
        _init()
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _current_device():
        raise ValueError(f"{name} is on {t.device}, which is not the current CUDA device")
    return dev


def _ints(dev, *vectors):
    """int32 vectors (tensor, entries at least, name), contiguous."""
    for t, n, name in vectors:
        if t.dtype is not _int32 or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor of at least {n} entries on the call's device")


def _rows(t, dtype, name, dev, shape=None):
    """Strides (token, head) of a [rows, heads, d] tensor, d contiguous."""
    st = t.stride()
    if len(st) != 3 or t.dtype is not dtype or st[2] != 1 or t.get_device() != dev or (
            shape is not None and t.shape != shape):
        want = "[rows, heads, d]" if shape is None else str(list(shape))
        raise ValueError(f"{name} must be a {want} tensor of type {dtype} on the call's device with d contiguous")
    return st[0], st[1]


def _pool(t, dtype, name, dev):
    """(shape, token stride, head stride) of a [blocks, block_size, Hk, d] pool."""
    st = t.stride()
    if len(st) != 4 or t.dtype is not dtype or st[3] != 1 or t.get_device() != dev:
        raise ValueError(f"{name} must be a [blocks, block_size, Hk, d] tensor of type {dtype} on the call's device "
                         "with d contiguous")
    shape = t.shape
    # (a block of one row has no token stride of its own)
    token = st[1] if shape[1] > 1 else st[0]
    if shape[0] > 1 and st[0] != shape[1] * token:
        raise ValueError(f"the blocks of {name} must follow one another with the token stride")
    return shape, token, st[2]


def _table(t, n_seqs, dev) -> int:
    shape = t.shape
    if t.dtype is not _int32 or len(shape) != 2 or shape[0] != n_seqs or shape[1] < 1 or (
            t.get_device() != dev or not t.is_contiguous()):
        raise ValueError("block_table must be a contiguous int32 [B, max_blocks] tensor on the call's device")
    return shape[1]


def _new(shape, dtype, like, stream):
    """An output or workspace that belongs to the call's stream."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


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
    call then takes nothing, every slot is -1 and every kv_len 0.
    ``pool_blocks`` bounds the block ids."""
    dev = _device_of(ctx_len, "ctx_len")
    n_seqs = ctx_len.numel()
    width = _table(block_table, n_seqs, dev)
    if slot_map is None:
        if n_tokens is None:
            raise ValueError("give slot_map or n_tokens")
        slot_map = _new(int(n_tokens), _int32, ctx_len, stream)
    elif n_tokens is None:
        n_tokens = slot_map.numel()
    if kv_len is None:
        kv_len = _new(n_seqs, _int32, ctx_len, stream)
    if n_left is None:
        n_left = _new(1, _int32, ctx_len, stream)
    _ints(dev, (ctx_len, 1, "ctx_len"), (new_off, n_seqs + 1, "new_off"), (free_blocks, 0, "free_blocks"),
          (n_free, 1, "n_free"), (slot_map, n_tokens, "slot_map"), (kv_len, n_seqs, "kv_len"), (n_left, 1, "n_left"))
    if status is not None:
        _ints(dev, (status, 1, "status"))
    if pool_blocks is None:
        pool_blocks = max(1, _INT32_MAX // max(1, int(block_size)))
    shape = _BlockShape(n_seqs, block_size, width, n_tokens, free_blocks.numel(), pool_blocks)
    rc = lib().sp_block_tables(shape, ctx_len.data_ptr(), new_off.data_ptr(), free_blocks.data_ptr(),
                               n_free.data_ptr(), block_table.data_ptr(), slot_map.data_ptr(), kv_len.data_ptr(),
                               n_left.data_ptr(), None if status is None else status.data_ptr(),
                               _raw_stream(dev) if stream is None else stream.cuda_stream)
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
    dev = _device_of(k, "k")
    dt = k.dtype
    code = _codes.get(dt)
    if code is None:
        raise ValueError("k must be bfloat16 or float16")
    shape = k.shape
    k_st, k_sh = _rows(k, dt, "k", dev)
    v_st, v_sh = _rows(v, dt, "v", dev, shape)
    n, hk, d = shape
    pool, kp_st, kp_sh = _pool(k_pool, dt, "k_pool", dev)
    v_pool_shape, vp_st, vp_sh = _pool(v_pool, dt, "v_pool", dev)
    if pool != v_pool_shape or pool[2] != hk or pool[3] != d:
        raise ValueError("k, v and the pools disagree on heads, head_dim or blocks")
    _ints(dev, (slot_map, n, "slot_map"))
    rotary = max_pos = 0
    if cos_sin is not None:
        if positions is None:
            raise ValueError("cos_sin needs positions")
        if cos_sin.dtype is not _float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous() or (
                cos_sin.get_device() != dev):
            raise ValueError("cos_sin must be a contiguous float32 [max_pos, rotary_dim] tensor on the call's device")
        max_pos, rotary = cos_sin.shape
        _ints(dev, (positions, n, "positions"))
    elif positions is not None:
        raise ValueError("positions need cos_sin")
    hq = q_st = q_sh = qo_st = qo_sh = 0
    if q is not None:
        q_st, q_sh = _rows(q, dt, "q", dev)
        q_shape = q.shape
        if q_shape[0] != n or q_shape[2] != d:
            raise ValueError("q and k disagree on tokens or head_dim")
        hq = q_shape[1]
        if q_out is None:
            q_out = _new(q_shape, dt, k, stream)
        qo_st, qo_sh = _rows(q_out, dt, "q_out", dev, q_shape)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if n_new is not None:
        _ints(dev, (n_new, 1, "n_new"))
    if status is not None:
        _ints(dev, (status, 1, "status"))
    if n == 0:
        return q_out
    rc = lib().sp_append_kv(
        _AppendShape(n, hq, hk, d, rotary, max_pos, code, 0, pool[0] * pool[1], q_st, q_sh, qo_st, qo_sh, k_st, k_sh,
                     v_st, v_sh, kp_st, kp_sh, vp_st, vp_sh),
        None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), slot_map.data_ptr(),
        None if positions is None else positions.data_ptr(), None if cos_sin is None else cos_sin.data_ptr(),
        None if n_new is None else n_new.data_ptr(), None if q is None else q_out.data_ptr(), k_pool.data_ptr(),
        v_pool.data_ptr(), None if status is None else status.data_ptr(),
        _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "sp_append_kv")
    return q_out


def _attention_shape(q, n_seqs, k_pool, dev, width=1, out=None, v_pool=None):
    dt = q.dtype
    code = _codes.get(dt)
    if code is None:
        raise ValueError("q must be bfloat16 or float16")
    q_st, q_sh = _rows(q, dt, "q", dev)
    n, hq, dq = shape = q.shape
    pool, k_st, k_sh = _pool(k_pool, dt, "k_pool", dev)
    nb, bs, hk, d = pool
    if dq != d:
        raise ValueError("q and the pools disagree on head_dim")
    o_st, o_sh = (hq * d, d) if out is None else _rows(out, dt, "out", dev, shape)
    v_st, v_sh = k_st, k_sh
    if v_pool is not None:
        v_pool_shape, v_st, v_sh = _pool(v_pool, dt, "v_pool", dev)
        if v_pool_shape != pool:
            raise ValueError("the pools disagree on heads, head_dim or blocks")
    return _PagedShape(n_seqs, hq, hk, d, code, bs, width, n, nb * bs, q_st, q_sh, o_st, o_sh, k_st, k_sh, v_st, v_sh)


def make_attention_workspace(q, n_seqs: int, k_pool, stream=None):
    """Workspace of paged_attention for queries of q's shape (its rows bound
    the new tokens of a call) of ``n_seqs`` requests over pools like
    ``k_pool``; calls that share one must be ordered."""
    import torch
    dev = _device_of(q, "q")
    shape = _attention_shape(q, int(n_seqs), k_pool, dev)
    n = _SZ()
    _check(lib().sp_paged_attention_workspace(shape, ctypes.byref(n)), "sp_paged_attention_workspace")
    ws = _new(n.value + 256, torch.uint8, q, stream)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n.value]
    _check(lib().sp_workspace_init(ws.data_ptr(), n.value,
                                   _raw_stream(dev) if stream is None else stream.cuda_stream), "sp_workspace_init")
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
    make_attention_workspace, with its status in device_status."""
    dev = _device_of(q, "q")
    n_seqs = kv_len.numel()
    _ints(dev, (kv_len, 1, "kv_len"), (q_off, n_seqs + 1, "q_off"))
    width = _table(block_table, n_seqs, dev)
    if out is None:
        out = _new(q.shape, q.dtype, q, stream)
    shape = _attention_shape(q, n_seqs, k_pool, dev, width, out, v_pool)
    if lse is not None and (lse.dtype is not _float32 or not lse.is_contiguous() or lse.shape != q.shape[:2]
                            or lse.get_device() != dev):
        raise ValueError("lse must be a contiguous float32 [T, Hq] tensor on the call's device")
    if shape.n_tokens == 0:
        return out
    if ws is None:
        ws = make_attention_workspace(q, n_seqs, k_pool, stream)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must come from make_attention_workspace on the call's device")
    rc = lib().sp_paged_attention(shape, _AttnParams(bool(causal), window, scale, spin_limit), q_off.data_ptr(),
                                  kv_len.data_ptr(), block_table.data_ptr(), q.data_ptr(), k_pool.data_ptr(),
                                  v_pool.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
                                  ws.data_ptr(), ws.nbytes, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "sp_paged_attention")
    return out
