"""Small cases of the paged-cache operators and the error bounds they are held to."""

import numpy as np

# half a unit in the last place, relative: the largest rounding error of a type
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def paged_case(seed, ctx, new, hq, hk, d, bs, dtype, spare_rows=0, q_gain=1.0, poison=True):
    """Tensors of an attention call: request b has ctx[b] + new[b] cached
    tokens, blocks shuffled over the pools. Rows that no request owns hold NaN
    when ``poison``. q has ``spare_rows`` rows behind the last request."""
    import torch
    rng = np.random.default_rng(seed)
    dt = torch_dtype(dtype)
    kv = [c + n for c, n in zip(ctx, new)]
    used = [-(-n // bs) for n in kv]
    blocks = sum(used) + 2
    perm = rng.permutation(blocks)
    table = np.full((len(kv), max(max(used), 1) + 1), -1, dtype=np.int32)   # (unused entries are invalid ids)
    pool = [np.full((blocks, bs, hk, d), np.nan if poison else 0.25, dtype=np.float32) for _ in range(2)]
    first = 0
    for b, n in enumerate(kv):
        ids = perm[first:first + used[b]]
        first += used[b]
        table[b, :used[b]] = ids
        for p in pool:
            rows = rng.standard_normal((n, hk, d), dtype=np.float32)
            flat = p.reshape(-1, hk, d)
            idx = (ids[:, None] * bs + np.arange(bs)).reshape(-1)[:n]
            flat[idx] = rows
    tokens = sum(new) + spare_rows
    q = rng.standard_normal((max(tokens, 1), hq, d), dtype=np.float32) * q_gain
    off = np.zeros(len(new) + 1, dtype=np.int32)
    off[1:] = np.cumsum(new)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return dict(q=dev(q).to(dt), q_off=dev(off), kv_len=dev(np.asarray(kv, dtype=np.int32)), table=dev(table),
                k_pool=dev(pool[0]).to(dt), v_pool=dev(pool[1]).to(dt))


def host(t):
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def attention_bounds(ref, kv_len, d, dtype):
    """Elementwise bounds of |out - ref| and |lse - ref|.

    With u the half step of the type and e = 2^-23 (twice the half step of
    fp32, for sums that are not rounded to nearest): a logit is a sum of d
    exact products in fp32, off by at most d e S with S = scale sum|q k|, and
    is scaled and shifted in three more roundings of values up to S + |m| <= 2 S,
    so |ds| <= (d + 8) e S. A weight's relative error is then |ds| (the
    reference m is the same in numerator and sum), 2^-22 of the exponential,
    and u of its own rounding for the product with the values; the sum of n of
    them adds n e, and the rescalings and joins of partial results at most 64 e.
    Numerator and sum both carry it: twice. 5 % covers the products of errors.
    The result's own rounding adds u |out|, or half the smallest subnormal
    (fp16: 2^-25)."""
    out, lse, weight, spread = ref
    u, e = HALF_STEP[dtype], 2.0 ** -23
    n = max(int(np.max(kv_len)), 1)
    ds = (d + 8) * e * spread
    rel = 1.05 * (2.0 * (ds + (n + 64) * e) + 2.0 ** -21 + u)
    tol_out = rel[..., None] * weight + u * np.abs(out) * 1.05 + 2.0 ** -25
    tol_lse = np.where(np.isfinite(lse), 1.05 * (ds + (n + 64) * e + 2.0 ** -22) + 8 * e * np.abs(np.where(np.isfinite(lse), lse, 0)), 0)
    return tol_out, tol_lse


def check_attention(out, lse, ref, kv_len, d, dtype, tokens):
    o = host(out)[:tokens]
    tol_out, tol_lse = attention_bounds(ref, kv_len, d, dtype)
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
