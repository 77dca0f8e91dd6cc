"""Small cases of the 4-bit cache and the error bounds they are held to."""

import numpy as np

from oracle import fp4_oracle
from tests.paged_cases import HALF_STEP, host, torch_dtype


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def fp4_case(seed, ctx, new, hq, hk, d, bs, dtype, spare_rows=0, q_gain=1.0, factor=(1.0, 1.0), poison=True):
    """Tensors of an attention call, as tests.paged_cases.paged_case makes them;
    rows that no request owns have NaN scales when ``poison``. The pools' values
    (with their factors) are in "k" and "v", float64."""
    rng = np.random.default_rng(seed)
    kv = [c + n for c, n in zip(ctx, new)]
    used = [-(-n // bs) for n in kv]
    blocks = sum(used) + 2
    perm = rng.permutation(blocks)
    # (unused entries are invalid ids; by rows this wide the call may be a long one, so that requests with many new
    # tokens go through 16 bits)
    table = np.full((len(kv), max(max(used), 1) + 90000 // bs), -1, dtype=np.int32)
    pools = []
    for f in factor:
        codes = rng.integers(0, 16, (blocks, bs, hk, d), dtype=np.uint8)
        scales = np.full((blocks, bs, hk, d // 16), 127 if poison else 40, dtype=np.uint8)
        pools.append((codes, scales))
    first = 0
    for b, n in enumerate(kv):
        ids = perm[first:first + used[b]]
        first += used[b]
        table[b, :used[b]] = ids
        idx = (ids[:, None] * bs + np.arange(bs)).reshape(-1)[:n]
        for codes, scales in pools:
            c, s = fp4_oracle.encode(rng.standard_normal((n, hk, d), dtype=np.float32))
            codes.reshape(-1, hk, d)[idx] = c
            scales.reshape(-1, hk, d // 16)[idx] = s
    tokens = sum(new) + spare_rows
    q = rng.standard_normal((max(tokens, 1), hq, d), dtype=np.float32) * q_gain
    off = np.zeros(len(new) + 1, dtype=np.int32)
    off[1:] = np.cumsum(new)
    packed = [fp4_oracle.pack(*p) for p in pools]
    return dict(q=dev(q).to(torch_dtype(dtype)), q_off=dev(off), kv_len=dev(np.asarray(kv, dtype=np.int32)),
                table=dev(table), k_pool=dev(packed[0]), v_pool=dev(packed[1]), k_scale=factor[0], v_scale=factor[1],
                k=fp4_oracle.values(packed[0], factor[0]), v=fp4_oracle.values(packed[1], factor[1]))


def attention_bounds(ref, kv_len, d, dtype, v_max):
    """tests.paged_cases.attention_bounds for the 4-bit cache. Products of 16-bit
    queries and values are exact there too, the scale's product with the factor is
    one rounding more (d + 9), and the weights are rounded to fp16 (half a step 2^-11, at
    most the type's) scaled so that the reference is 2^6: one below 2^-14 is off by up
    to 2^-25 of its own, 2^-31 of the reference, which is at most the sum of the weights: n
    of them move the result by n 2^-31 of the largest value. The value's factor adds
    one rounding (in the 64 e)."""
    out, lse, weight, spread = ref
    u, e = HALF_STEP[dtype], 2.0 ** -23
    n = max(int(np.max(kv_len)), 1)
    ds = (d + 9) * e * spread
    rel = 1.05 * (2.0 * (ds + (n + 64) * e) + 2.0 ** -21 + u)
    tol_out = rel[..., None] * weight + u * np.abs(out) * 1.05 + 2.0 ** -25 + 1.05 * n * 2.0 ** -31 * v_max
    safe = np.where(np.isfinite(lse), lse, 0)
    tol_lse = np.where(np.isfinite(lse), 1.05 * (ds + (n + 64) * e + 2.0 ** -22) + 8 * e * np.abs(safe), 0)
    return tol_out, tol_lse


def check_attention(out, lse, ref, kv_len, d, dtype, tokens, v_max):
    o = host(out)[:tokens]
    tol_out, tol_lse = attention_bounds(ref, kv_len, d, dtype, v_max)
    assert np.isfinite(o).all()
    excess = np.abs(o - ref[0][:tokens]) - tol_out[:tokens]
    assert excess.max(initial=-1.0) <= 0, f"out is {excess.max()} over its bound"
    if lse is not None:
        s = host(lse)[:tokens]
        r = ref[1][:tokens]
        none = np.isneginf(r)
        assert np.array_equal(np.isneginf(s), none)
        gap = np.abs(np.where(none, 0, s) - np.where(none, 0, r)) - tol_lse[:tokens]
        assert gap.max(initial=-1.0) <= 0, f"lse is {gap.max()} over its bound"
