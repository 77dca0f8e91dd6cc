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

from . import _SZ, _check, _ptr, _stream, lib


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


def _on(device, t, name):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")


def _device_of(t, name):
    """The device of a call: that of its first tensor, which has to be the
    current CUDA device (the library launches there)."""
    import torch
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, which is not the current CUDA device")
    return t.device


def _ints(t, n, name, device):
    """An int32 vector of at least n entries, contiguous."""
    import torch
    if t.dtype is not torch.int32 or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name} must be a contiguous int32 tensor of at least {n} entries")
    _on(device, t, name)


def _dtype_code(t, name):
    import torch
    if t.dtype is torch.bfloat16:
        return 0
    if t.dtype is torch.float16:
        return 1
    raise ValueError(f"{name} must be bfloat16 or float16")


def _rows(t, dtype, name, device, shape=None):
    """Strides (token, head) of a [rows, heads, d] tensor, d contiguous."""
    if t.dim() != 3 or t.dtype is not dtype or t.stride(2) != 1 or (shape is not None and t.shape != shape):
        want = "[rows, heads, d]" if shape is None else str(list(shape))
        raise ValueError(f"{name} must be a {want} tensor of type {dtype} with d contiguous")
    _on(device, t, name)
    return t.stride(0), t.stride(1)


def _pool(t, dtype, name, device):
    """(blocks, block_size, Hk, d, token stride, head stride) of a pool."""
    if t.dim() != 4 or t.dtype is not dtype or t.stride(3) != 1:
        raise ValueError(f"{name} must be a [blocks, block_size, Hk, d] tensor of type {dtype} with d contiguous")
    nb, bs, hk, d = t.shape
    # (a block of one row has no token stride of its own)
    st = t.stride(1) if bs > 1 else t.stride(0)
    if nb > 1 and t.stride(0) != bs * st:
        raise ValueError(f"the blocks of {name} must follow one another with the token stride")
    _on(device, t, name)
    return nb, bs, hk, d, st, t.stride(2)


def _table(t, n_seqs, device):
    import torch
    if t.dtype is not torch.int32 or t.dim() != 2 or t.shape[0] != n_seqs or t.shape[1] < 1 or not t.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 [B, max_blocks] tensor")
    _on(device, t, "block_table")


def _new(shape, dtype, device, stream):
    """An output or workspace that belongs to the call's stream."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


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
    import torch
    n_seqs = ctx_len.numel()
    dev = _device_of(ctx_len, "ctx_len")
    _ints(ctx_len, 1, "ctx_len", dev)
    _ints(new_off, n_seqs + 1, "new_off", dev)
    _ints(free_blocks, 0, "free_blocks", dev)
    _ints(n_free, 1, "n_free", dev)
    _table(block_table, n_seqs, dev)
    if slot_map is None:
        if n_tokens is None:
            raise ValueError("give slot_map or n_tokens")
        slot_map = _new(int(n_tokens), torch.int32, dev, stream)
    elif n_tokens is None:
        n_tokens = slot_map.numel()
    _ints(slot_map, n_tokens, "slot_map", dev)
    if kv_len is None:
        kv_len = _new(n_seqs, torch.int32, dev, stream)
    _ints(kv_len, n_seqs, "kv_len", dev)
    if n_left is None:
        n_left = _new(1, torch.int32, dev, stream)
    _ints(n_left, 1, "n_left", dev)
    if status is not None:
        _ints(status, 1, "status", dev)
    if pool_blocks is None:
        pool_blocks = max(1, _INT32_MAX // max(1, int(block_size)))
    shape = _BlockShape(n_seqs, int(block_size), block_table.shape[1], int(n_tokens), free_blocks.numel(),
                        int(pool_blocks))
    _check(lib().sp_block_tables(ctypes.byref(shape), ctx_len.data_ptr(), new_off.data_ptr(), free_blocks.data_ptr(),
                                 n_free.data_ptr(), block_table.data_ptr(), slot_map.data_ptr(), kv_len.data_ptr(),
                                 n_left.data_ptr(), _ptr(status), _stream(stream)), "sp_block_tables")
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
    n, hk, d = k.shape if k.dim() == 3 else (0, 0, 0)
    dev = _device_of(k, "k")
    code = _dtype_code(k, "k")
    dt = k.dtype
    k_st, k_sh = _rows(k, dt, "k", dev)
    v_st, v_sh = _rows(v, dt, "v", dev, k.shape)
    _ints(slot_map, n, "slot_map", dev)
    nb, bs, khk, kd, kp_st, kp_sh = _pool(k_pool, dt, "k_pool", dev)
    vnb, vbs, vhk, vd, vp_st, vp_sh = _pool(v_pool, dt, "v_pool", dev)
    if (nb, bs, khk, kd) != (vnb, vbs, vhk, vd) or khk != hk or kd != d:
        raise ValueError("k, v and the pools disagree on heads, head_dim or blocks")
    rotary = max_pos = 0
    if cos_sin is not None:
        import torch
        if cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be a contiguous float32 [max_pos, rotary_dim] tensor")
        _on(dev, cos_sin, "cos_sin")
        if positions is None:
            raise ValueError("cos_sin needs positions")
        max_pos, rotary = cos_sin.shape
        _ints(positions, n, "positions", dev)
    elif positions is not None:
        raise ValueError("positions need cos_sin")
    hq = q_st = q_sh = qo_st = qo_sh = 0
    if q is not None:
        q_st, q_sh = _rows(q, dt, "q", dev)
        if q.shape[0] != n or q.shape[2] != d:
            raise ValueError("q and k disagree on tokens or head_dim")
        hq = q.shape[1]
        if q_out is None:
            q_out = _new(q.shape, dt, dev, stream)
        qo_st, qo_sh = _rows(q_out, dt, "q_out", dev, q.shape)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if n_new is not None:
        _ints(n_new, 1, "n_new", dev)
    if status is not None:
        _ints(status, 1, "status", dev)
    if n == 0:
        return q_out
    shape = _AppendShape(n, hq, hk, d, rotary, max_pos, code, 0, nb * bs, q_st, q_sh, qo_st, qo_sh, k_st, k_sh, v_st,
                         v_sh, kp_st, kp_sh, vp_st, vp_sh)
    _check(lib().sp_append_kv(ctypes.byref(shape), _ptr(q), k.data_ptr(), v.data_ptr(), slot_map.data_ptr(),
                              _ptr(positions), _ptr(cos_sin), _ptr(n_new), _ptr(q_out), k_pool.data_ptr(),
                              v_pool.data_ptr(), _ptr(status), _stream(stream)), "sp_append_kv")
    return q_out


def _attention_shape(q, n_seqs, k_pool, device, table_stride=1, out=None, v_pool=None):
    code = _dtype_code(q, "q")
    dt = q.dtype
    q_st, q_sh = _rows(q, dt, "q", device)
    nb, bs, hk, d, k_st, k_sh = _pool(k_pool, dt, "k_pool", device)
    n, hq, dq = q.shape
    if dq != d:
        raise ValueError("q and the pools disagree on head_dim")
    o_st, o_sh = (hq * d, d) if out is None else _rows(out, dt, "out", device, q.shape)
    v_st, v_sh = k_st, k_sh
    if v_pool is not None:
        vnb, vbs, vhk, vd, v_st, v_sh = _pool(v_pool, dt, "v_pool", device)
        if (vnb, vbs, vhk, vd) != (nb, bs, hk, d):
            raise ValueError("the pools disagree on heads, head_dim or blocks")
    return _PagedShape(n_seqs, hq, hk, d, code, bs, table_stride, n, nb * bs, q_st, q_sh, o_st, o_sh, k_st, k_sh,
                       v_st, v_sh)


def make_attention_workspace(q, n_seqs: int, k_pool, stream=None):
    """Workspace of paged_attention for queries of q's shape (its rows bound
    the new tokens of a call) of ``n_seqs`` requests over pools like
    ``k_pool``; calls that share one must be ordered."""
    import torch
    dev = _device_of(q, "q")
    shape = _attention_shape(q, int(n_seqs), k_pool, dev)
    n = _SZ()
    _check(lib().sp_paged_attention_workspace(ctypes.byref(shape), ctypes.byref(n)), "sp_paged_attention_workspace")
    ws = _new(n.value + 256, torch.uint8, dev, stream)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n.value]
    _check(lib().sp_workspace_init(ws.data_ptr(), n.value, _stream(stream)), "sp_workspace_init")
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
    import torch
    n_seqs = kv_len.numel()
    dev = _device_of(q, "q")
    _ints(kv_len, 1, "kv_len", dev)
    _ints(q_off, n_seqs + 1, "q_off", dev)
    _table(block_table, n_seqs, dev)
    if out is None:
        out = _new(q.shape, q.dtype, dev, stream)
    shape = _attention_shape(q, n_seqs, k_pool, dev, block_table.shape[1], out, v_pool)
    if lse is not None:
        if lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.shape != q.shape[:2]:
            raise ValueError("lse must be a contiguous float32 [T, Hq] tensor")
        _on(dev, lse, "lse")
    if shape.n_tokens == 0:
        return out
    if ws is None:
        ws = make_attention_workspace(q, n_seqs, k_pool, stream)
    _on(dev, ws, "ws")
    params = _AttnParams(int(bool(causal)), int(window), float(scale), int(spin_limit))
    _check(lib().sp_paged_attention(ctypes.byref(shape), ctypes.byref(params), q_off.data_ptr(), kv_len.data_ptr(),
                                    block_table.data_ptr(), q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
                                    out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(), _stream(stream)),
           "sp_paged_attention")
    return out
