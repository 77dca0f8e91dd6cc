"""Attention from the 4-bit rows themselves: its weights' 11 bits, requests among
others, batches whose layout leaves 24 bits."""

import numpy as np
import pytest

from oracle import paged_oracle
from tests.fp4_cases import attention_bounds, dev, fp4_case
from tests.paged_cases import HALF_STEP, host

pytestmark = pytest.mark.gpu


def attend(c, **more):
    import torch

    import speculative_prefill_token_gb300 as sp
    ws = sp.make_attention_fp4_workspace(c["q"], c["kv_len"].numel(), c["k_pool"], kv_tokens=0)
    lse = torch.full(c["q"].shape[:2], 7.0, dtype=torch.float32, device="cuda")
    out = sp.paged_attention_fp4(c["q"], c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"], k_scale=c["k_scale"],
                                 v_scale=c["v_scale"], lse=lse, ws=ws, **more)
    assert sp.device_status(ws) == 0
    return out, lse


def reference(c, window=0):
    return paged_oracle.paged_attention(host(c["q"]), host(c["q_off"]), host(c["kv_len"]), host(c["table"]),
                                        np.nan_to_num(c["k"]), np.nan_to_num(c["v"]), window=window)


def bound_of_fp16_weights(c, ref):
    """attention_bounds with the weights' own half step, 2^-11, in place of the result's type's: a bf16 result is
    rounded once, by its half step of itself."""
    d, v_max = c["q"].shape[2], float(np.nanmax(np.abs(c["v"])))
    tol, _ = attention_bounds(ref, host(c["kv_len"]), d, "fp16", v_max)
    return tol + (HALF_STEP["bf16"] - HALF_STEP["fp16"]) * np.abs(ref[0]) * 1.05


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ctx,new", [([511, 40, 0], [1, 1, 1]), ([30011, 77], [8, 1]), ([300, 0], [150, 70])])
def test_weights_have_11_bits(d, ctx, new):
    c = fp4_case(d, ctx, new, 8, 2, d, 32, "bf16", factor=(0.5, 2.0))
    ref = reference(c)
    out, _ = attend(c)
    excess = np.abs(host(out) - ref[0]) - bound_of_fp16_weights(c, ref)
    assert excess.max() <= 0


@pytest.mark.parametrize("d", [64, 256])
def test_a_request_among_other_requests(d):
    """Where an item is cut depends on the whole batch: a request's result keeps to its bound whatever is beside it, and
    the same batch gives the same bits."""
    import torch
    rng = np.random.default_rng(d)
    base = fp4_case(d, [7000, 500, 3, 20000, 0], [2, 1, 1, 1, 9], 8, 2, d, 16, "bf16")
    ref = reference(base)
    tol = bound_of_fp16_weights(base, ref)
    off = host(base["q_off"])
    seen = []
    for others in ([1, 2, 3, 4], [], [3], [1, 1, 1, 4, 4], [3] * 20, [2] * 70):
        order = rng.permutation([0] + others)
        new = [off[b + 1] - off[b] for b in order]
        rows = np.concatenate([np.arange(off[b], off[b + 1]) for b in order])
        c = dict(base, q=base["q"][dev(rows)], kv_len=base["kv_len"][dev(order)], table=base["table"][dev(order)].contiguous(),
                 q_off=dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)))
        out, lse = attend(c)
        again = attend(c)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
        assert (np.abs(host(out) - ref[0][rows]) <= tol[rows]).all()
        seen.append(out[dev(np.flatnonzero(rows < off[1]))])
    assert all(len(x) == 2 for x in seen)


def test_a_layout_that_leaves_24_bits():
    """16 decode steps of 65,536 heads: the costs of all items are more than a warp's layout adds up."""
    import torch

    import speculative_prefill_token_gb300 as sp
    hk, d, bs, batch, item_cost = 65536, 64, 8, 16, 16
    kv = np.array([0] + [1 + 3 * i % 24 for i in range(1, batch)], dtype=np.int32)
    held = -(-kv // bs)
    assert hk * ((kv > 0).sum() + batch * item_cost) > 1 << 24
    gen = torch.Generator(device="cuda").manual_seed(0)
    blocks = int(held.sum())
    pools = []
    for _ in range(2):
        pool = torch.randint(0, 256, (blocks, hk, 1, 9 * d // 2), dtype=torch.uint8, device="cuda", generator=gen)
        pool[..., 4 * d:] = pool[..., 4 * d:] % 21 + 40     # scales from 1/4 to 1.5
        pools.append(pool)
    table = np.full((batch, 4), -1, dtype=np.int32)
    ids = np.random.default_rng(0).permutation(blocks)
    for b in range(batch):
        table[b, :held[b]], ids = ids[:held[b]], ids[held[b]:]
    q = torch.randn(batch, hk, d, device="cuda", generator=gen).bfloat16()
    off = dev(np.arange(batch + 1, dtype=np.int32))

    def call(heads):
        out = torch.full((batch, heads.stop - heads.start, d), 7.0, device="cuda").bfloat16()
        lse = torch.full(out.shape[:2], 7.0, device="cuda")
        parts = [p[:, heads] for p in pools]
        ws = sp.make_attention_fp4_workspace(q[:, heads], batch, parts[0], max_new=1)
        sp.paged_attention_fp4(q[:, heads], off, dev(kv), dev(table), *parts, out=out, lse=lse, max_new=1, ws=ws)
        assert sp.device_status(ws) == 0
        return out, lse

    out, lse = call(slice(0, hk))
    # the same by a quarter of the heads at a time, which a warp lays out
    for h in range(0, hk, hk // 4):
        part = call(slice(h, h + hk // 4))
        assert torch.equal(part[0], out[:, h:h + hk // 4]) and torch.equal(part[1], lse[:, h:h + hk // 4])
    some = [0, 1, 777, 40000, hk - 1]
    k, v = (host(sp.unpack_fp4(p[:, some].contiguous())) for p in pools)
    ref = paged_oracle.paged_attention(host(q[:, some]), np.arange(batch + 1), kv, table, k, v)
    c = dict(q=q, kv_len=dev(kv), v=v)
    assert (np.abs(host(out[:, some]) - ref[0]) <= bound_of_fp16_weights(c, ref)).all()
    assert np.array_equal(np.isneginf(host(lse[:, some])), np.isneginf(ref[1]))
