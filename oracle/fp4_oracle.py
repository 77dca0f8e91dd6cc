"""Restatement of the 4-bit cache and of the page operators from their
definitions in include/specprefill.h: rows to codes and scales (the definition's
32-bit operations, each rounded), codes and scales to float64 values, forks,
frees and copies by plain loops. Test infrastructure."""

import numpy as np

NUMBERS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_values():
    """The 128 e4m3 numbers of a clear sign bit (the last one is NaN)."""
    byte = np.arange(128)
    e, m = byte >> 3, byte & 7
    v = np.where(e == 0, m / 512.0, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[127] = np.nan
    return v


def nearest(x, table):
    """Index of the nearest entry of an increasing table for x >= 0, ties to the
    even index, at most the last entry (in exact arithmetic: float64 holds
    entries, their middles and x)."""
    x = np.asarray(x, dtype=np.float64)
    middle = (table[1:] + table[:-1]) / 2
    low = np.searchsorted(middle, x, side="left")     # middles below x
    tie = (low < len(middle)) & (x == middle[np.minimum(low, len(middle) - 1)])
    return np.where(tie & (low % 2 == 1), low + 1, low)


def encode(x, factor=1.0):
    """(codes, scale bytes) of fp32 rows [..., d]: codes [..., d] with bit 3 the
    sign, scales [..., d / 16]."""
    x = np.asarray(x, dtype=np.float32)
    y = (x * (np.float32(1) / np.float32(factor))).reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    with np.errstate(invalid="ignore"):
        top = np.abs(y).max(-1)
        bad = ~np.isfinite(y).all(-1)
        byte = np.maximum(nearest(np.where(bad, 0, top / np.float32(6.0)), scale_values()[:127]), 1)
        s = scale_values()[byte].astype(np.float32)
        r = np.where(bad[..., None], 0, y / s[..., None])
    code = nearest(np.abs(r), NUMBERS) + 8 * (np.signbit(r) & ~bad[..., None])
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 127, byte).astype(np.uint8)


def decode(codes, scales):
    """Values [..., d] in float64."""
    v = np.concatenate([NUMBERS, -NUMBERS])[codes]
    return v * np.repeat(scale_values()[scales & 127] * np.where(scales > 127, -1, 1), 16, axis=-1)


def pack(codes, scales):
    """Rows [blocks, bs, Hk, d] of codes and their scales as a pool
    [blocks, Hk, bs / 8, 9 d / 2] of bytes."""
    blocks, bs, hk, d = codes.shape
    c = (codes[..., 0::2] | codes[..., 1::2] << 4).transpose(0, 2, 1, 3).reshape(blocks, hk, bs // 8, 4 * d)
    s = scales.transpose(0, 2, 1, 3).reshape(blocks, hk, bs // 8, d // 2)
    return np.concatenate([c, s], -1).astype(np.uint8)


def unpack(pool):
    """(codes, scales) as `pack` takes them."""
    blocks, hk, groups, width = pool.shape
    d = width * 2 // 9
    c = pool[..., :4 * d].reshape(blocks, hk, groups * 8, d // 2).transpose(0, 2, 1, 3)
    s = pool[..., 4 * d:].reshape(blocks, hk, groups * 8, d // 16).transpose(0, 2, 1, 3)
    return np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], d), s


def values(pool, factor=1.0):
    """[blocks, bs, Hk, d] in float64."""
    return decode(*unpack(pool)) * factor


def rotate32(x, positions, cos_sin):
    """The rotate-half rotation in the definition's 32-bit operations."""
    x = np.array(x, dtype=np.float32)
    half = cos_sin.shape[1] // 2
    turn = np.asarray(cos_sin, dtype=np.float32)[np.asarray(positions)][:, None, :]
    cos, sin = turn[..., :half], turn[..., half:]
    a, b = x[..., :half].copy(), x[..., half:2 * half].copy()
    x[..., :half] = a * cos - b * sin
    x[..., half:2 * half] = b * cos + a * sin
    return x


def fork_blocks(src, dst, ctx_len, table, shared, free, n_free, bs):
    """(kv_len, copy_src, copy_dst, n_left, table, shared), or None when the list
    is too short."""
    table, shared, kv = np.array(table), np.array(shared), np.array(ctx_len)
    free = [int(x) for x in free[:n_free]]
    copy = np.full((2, len(src)), -1)
    for i, (s, t) in enumerate(zip(src, dst)):
        if s < 0:
            continue
        n = int(ctx_len[s])
        kv[t] = n
        for k in range(n // bs):
            table[t, k] = table[s, k]
            shared[table[s, k]] += 1
        if n % bs:
            if not free:
                return None
            copy[:, i] = table[s, n // bs], free.pop()
            table[t, n // bs] = copy[1, i]
    return kv, copy[0], copy[1], len(free), table, shared


def free_blocks(ctx_len, new_len, table, shared, free, n_free, bs):
    """(kv_len, n_left, shared, free), or None when a block is let go too often
    or the list is too short."""
    shared, free = np.array(shared), np.array(free)
    holders = shared + 1
    gone = set()
    for b in range(len(ctx_len)):
        for k in range(-(-int(new_len[b]) // bs), -(-int(ctx_len[b]) // bs)):
            i = int(table[b, k])
            holders[i] -= 1
            if holders[i] < 0:
                return None
            if holders[i] == 0:
                gone.add(i)
    if n_free + len(gone) > len(free):
        return None
    shared = np.where(holders > 0, holders - 1, 0)
    free[n_free:n_free + len(gone)] = sorted(gone)
    return np.array(new_len), n_free + len(gone), shared, free
