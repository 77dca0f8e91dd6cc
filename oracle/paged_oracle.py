"""Float64 restatement of the paged-cache operators (block tables and slots,
rotation and store, attention over a paged cache), from their definitions in
include/specprefill.h. Plain loops over requests; test infrastructure."""

import numpy as np


def block_tables(ctx_len, new_off, free_blocks, n_free, table, block_size, n_tokens):
    """(table, slot_map, kv_len, n_left), or None when the free list is too
    short. The inputs are not changed."""
    table = np.array(table, dtype=np.int64)
    free = [int(x) for x in np.asarray(free_blocks)[:n_free]]
    slots = np.full(n_tokens, -1, dtype=np.int64)
    for b, ctx in enumerate(ctx_len):
        for t in range(int(new_off[b]), int(new_off[b + 1])):
            p = int(ctx) + t - int(new_off[b])
            if p % block_size == 0:
                if not free:
                    return None
                table[b, p // block_size] = free.pop()
            slots[t] = table[b, p // block_size] * block_size + p % block_size
    new = np.diff(np.asarray(new_off, dtype=np.int64))
    return table, slots, np.asarray(ctx_len, dtype=np.int64) + new, len(free)


def rotate(x, positions, cos_sin):
    """Rotate-half rotation of x [T, H, d] (float64) by the table's rows."""
    x = np.array(x, dtype=np.float64)
    half = cos_sin.shape[1] // 2
    turn = np.asarray(cos_sin, dtype=np.float64)[np.asarray(positions)][:, None, :]
    cos, sin = turn[..., :half], turn[..., half:]
    a, b = x[..., :half].copy(), x[..., half:2 * half].copy()
    x[..., :half] = a * cos - b * sin
    x[..., half:2 * half] = b * cos + a * sin
    return x


def paged_attention(q, q_off, kv_len, table, k_pool, v_pool, causal=True, window=0, scale=None):
    """(out, lse, weight, spread): out [T, Hq, d] and lse [T, Hq] in float64;
    weight[t, h] = sum_j p_j |v_j| (elementwise, [T, Hq, d]) and spread [T, Hq]
    = the largest scale * sum_i |q_i k_i| of a seen key, for error bounds.
    Pools are [blocks, block_size, Hk, d]; rows that nothing sees are unused."""
    q = np.asarray(q, dtype=np.float64)
    n_tok, hq, d = q.shape
    bs, hk = k_pool.shape[1], k_pool.shape[2]
    g = hq // hk
    scale = 1.0 / np.sqrt(d) if not scale else scale
    out = np.zeros((n_tok, hq, d))
    weight = np.zeros((n_tok, hq, d))
    lse = np.full((n_tok, hq), -np.inf)
    spread = np.zeros((n_tok, hq))
    for b, kv in enumerate(int(x) for x in kv_len):
        lo, hi = int(q_off[b]), int(q_off[b + 1])
        if hi == lo or kv == 0:
            continue
        pages = np.asarray(table[b, :-(-kv // bs)], dtype=np.int64)
        k = np.asarray(k_pool[pages], dtype=np.float64).reshape(-1, hk, d)[:kv]
        v = np.asarray(v_pool[pages], dtype=np.float64).reshape(-1, hk, d)[:kv]
        pos = kv - (hi - lo) + np.arange(hi - lo)
        j = np.arange(kv)
        seen = np.ones((hi - lo, kv), dtype=bool)
        if causal:
            seen = j <= pos[:, None]
            if window:
                seen &= j > pos[:, None] - window
        rows = seen.any(1)
        for h in range(hq):
            kh, vh = k[:, h // g], v[:, h // g]
            s = (q[lo:hi, h] @ kh.T) * scale
            s = np.where(seen, s, -np.inf)
            m = np.where(rows, s.max(1, initial=-np.inf), 0.0)
            p = np.where(seen, np.exp(s - m[:, None]), 0.0)
            total = p.sum(1)
            safe = np.where(rows, total, 1.0)
            out[lo:hi, h] = np.where(rows[:, None], p @ vh / safe[:, None], 0.0)
            weight[lo:hi, h] = np.where(rows[:, None], p @ np.abs(vh) / safe[:, None], 0.0)
            lse[lo:hi, h] = np.where(rows, m + np.log(safe), -np.inf)
            mags = (np.abs(q[lo:hi, h]) @ np.abs(kh).T) * scale
            spread[lo:hi, h] = np.where(seen, mags, 0.0).max(1, initial=0.0)
    return out, lse, weight, spread
