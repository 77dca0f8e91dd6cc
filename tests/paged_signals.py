"""Attention cases in which every small group of cached keys carries weight.

A bound that grows with the number of keys cannot see a key tile that was lost
among hundreds. Here some keys, the signals, point along the queries, so that
they hold nearly all of the softmax's mass in equal shares, and each has a large
value in one column of its own (or shared with few others): without one of them
its column loses a large part of itself. The bounds count what a sum by tiles
and parts goes through, not the number of keys."""

import numpy as np

from tests.paged_cases import HALF_STEP, host, torch_dtype

GAIN = 14.0     # logit of a signal; the other keys' are some units around 0
LOUD = 16.0     # value of a signal in its column; the other values' are some units
TILE = 128      # keys of a tile


def signal_arrays(seed, ctx, new, hq, hk, d, bs, dtype, every=16):
    """float32 arrays with values of the type: signals at a random place of every
    `every` keys, at both edges of each tile, and at all new tokens (of the
    last 16 of them at most)."""
    import torch
    rng = np.random.default_rng(seed)
    kv = [c + n for c, n in zip(ctx, new)]
    used = [-(-n // bs) for n in kv]
    blocks = sum(used) + 2
    perm = rng.permutation(blocks)
    table = np.full((len(kv), max(max(used), 1) + 1), -1, dtype=np.int32)
    k_pool, v_pool = [np.full((blocks, bs, hk, d), np.nan, dtype=np.float32) for _ in range(2)]
    along = rng.standard_normal((hk, d)).astype(np.float32)
    along /= np.linalg.norm(along, axis=1, keepdims=True)
    first = 0
    for b, n in enumerate(kv):
        ids = perm[first:first + used[b]]
        first += used[b]
        table[b, :used[b]] = ids
        k = 0.5 * rng.standard_normal((n, hk, d), dtype=np.float32)
        v = 0.5 * rng.standard_normal((n, hk, d), dtype=np.float32)
        at = np.arange(0, n, every)
        at = np.concatenate([np.minimum(at + rng.integers(0, every, at.size), n - 1), np.arange(0, n, TILE),
                             np.arange(TILE - 1, n, TILE), np.arange(max(ctx[b] - 1, n - 16, 0), n)])
        at = np.unique(at)
        # the noise of a signal across its direction only: all signals weigh alike
        k[at] -= (k[at] * along).sum(-1, keepdims=True) * along
        k[at] += along * d ** 0.25
        v[at, :, np.arange(at.size) % d] = LOUD
        idx = (ids[:, None] * bs + np.arange(bs)).reshape(-1)[:n]
        k_pool.reshape(-1, hk, d)[idx] = k
        v_pool.reshape(-1, hk, d)[idx] = v
    q = 0.5 * rng.standard_normal((sum(new), hk, hq // hk, d), dtype=np.float32)
    q -= (q * along[:, None]).sum(-1, keepdims=True) * along[:, None]
    q += along[:, None] * GAIN * d ** 0.25
    rounded = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(torch_dtype(dtype)).float().numpy()  # noqa: E731
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(q=rounded(q.reshape(-1, hq, d)), q_off=off, kv_len=np.asarray(kv, dtype=np.int32), table=table,
                k_pool=rounded(k_pool), v_pool=rounded(v_pool))


def tiled_bounds(ref, kv_len, d, dtype):
    """Elementwise bounds of |out - ref| and |lse - ref|.

    u and e as in attention_bounds, and the same errors of a logit, ds, of an
    exponential, 2^-22, and of a weight, u. A value is added to at most TILE
    others of its tile, then with at most `tiles` tiles of its part, then with at
    most as many parts: a sum of fp32 steps of TILE + 2 tiles roundings of e each,
    whatever the number of keys, and 64 more for rescalings and joins. Numerator
    and sum both carry ds and the depth. The result's own rounding adds u |out|,
    or half the smallest subnormal (fp16: 2^-25)."""
    out, lse, weight, spread = ref
    u, e = HALF_STEP[dtype], 2.0 ** -23
    depth = TILE + 2 * -(-max(int(np.max(kv_len)), 1) // TILE) + 64
    ds = (d + 8) * e * spread
    rel = 1.05 * (2.0 * (ds + depth * e) + 2.0 ** -21 + u)
    finite = np.isfinite(lse)
    tol_lse = np.where(finite, 1.05 * (ds + depth * e + 2.0 ** -22) + 8 * e * np.abs(np.where(finite, lse, 0)), 0)
    return rel[..., None] * weight + u * np.abs(out) * 1.05 + 2.0 ** -25, tol_lse


def check_signals(out, lse, ref, kv_len, d, dtype):
    """out and lse (tensors or arrays) within the bounds."""
    o, s = [host(x) if hasattr(x, "cpu") else np.asarray(x, dtype=np.float64) for x in (out, lse)]
    tol_out, tol_lse = tiled_bounds(ref, kv_len, d, dtype)
    assert np.isfinite(o).all()
    excess = (np.abs(o - ref[0]) - tol_out).max(initial=-1.0)
    assert excess <= 0, f"out is {excess} over its bound"
    none = np.isneginf(ref[1])
    assert np.array_equal(np.isneginf(s), none)
    excess = (np.abs(np.where(none, 0, s) - np.where(none, 0, ref[1])) - tol_lse).max(initial=-1.0)
    assert excess <= 0, f"lse is {excess} over its bound"
