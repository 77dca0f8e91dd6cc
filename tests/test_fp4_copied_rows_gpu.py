"""Requests of the 4-bit attention that are read through the 16-bit copy in the
workspace. Every test looks for a row of the cache in the workspace, so that it
fails when its request no longer goes that way."""

import numpy as np
import pytest

from oracle import paged_oracle
from tests.fp4_cases import check_attention, dev, fp4_case
from tests.paged_cases import host

pytestmark = pytest.mark.gpu


def held_in_16_bits(c, ws, request, token):
    """Whether the workspace holds the key of a cached token (the pools' values, without their factor)."""
    import speculative_prefill_token_gb300 as sp
    bs = c["k_pool"].shape[2] * 8
    slot = int(c["table"][request, token // bs]) * bs + token % bs
    row = sp.unpack_fp4(c["k_pool"], c["q"].dtype, slots=dev(np.array([slot], dtype=np.int32)))[0, 0, :64]
    return bool((ws.buffer.view(c["q"].dtype).view(-1, 64) == row).all(1).any())


def attend(c, copied=(), causal=True, window=0, scale=0.0, max_new=None, kv_tokens=None, ws=None, **more):
    """(out, lse, status); the requests in ``copied`` have gone through the copy, decode steps have not."""
    import torch

    import speculative_prefill_token_gb300 as sp
    if ws is None:
        ws = sp.make_attention_fp4_workspace(c["q"], c["kv_len"].numel(), c["k_pool"], max_new=max_new, kv_tokens=kv_tokens)
    ws.buffer[256:].fill_(0xff)   # (what lies behind a copied request's end is no number)
    out = torch.full_like(c["q"], 7.0)
    lse = torch.full(c["q"].shape[:2], 7.0, dtype=torch.float32, device="cuda")
    sp.paged_attention_fp4(c["q"], c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"], causal=causal,
                           window=window, scale=scale, k_scale=c["k_scale"], v_scale=c["v_scale"], out=out, lse=lse,
                           max_new=max_new, ws=ws, **more)
    new = np.diff(host(c["q_off"]))
    for b in copied:
        assert held_in_16_bits(c, ws, b, int(c["kv_len"][b]) - 1), b
    for b in np.flatnonzero(new == 1)[:2]:
        assert not held_in_16_bits(c, ws, b, int(c["kv_len"][b]) - 1), b
    return out, lse, sp.device_status(ws)


def check(c, dtype, copied, causal=True, window=0, table=None, **more):
    out, lse, status = attend(c, copied, causal, window, **more)
    assert status == 0
    ref = paged_oracle.paged_attention(host(c["q"]), host(c["q_off"]), host(c["kv_len"]), host(c["table"]) if table is None else table,
                                       np.nan_to_num(c["k"]), np.nan_to_num(c["v"]), causal, window)
    check_attention(out, lse, ref, host(c["kv_len"]), c["q"].shape[2], dtype, int(c["q_off"][-1]),
                    float(np.nanmax(np.abs(c["v"]))))


@pytest.mark.parametrize("window", [0, 250])
@pytest.mark.parametrize("batch", [3, 70, 400])
@pytest.mark.parametrize("longer", [1, 300])
def test_a_context_longer_than_its_pool_beside_a_chunk(batch, longer, window):
    """A request whose table row names its blocks over and over has more cached tokens than the pool: its
    rows, few or many, are computed from the 4-bit rows, the others' as ever."""
    bs = 16
    new = [1] * batch
    new[0], new[2] = longer, 200
    ctx = [40 + i % 5 for i in range(batch)]
    ctx[0] = 400 - longer
    c = fp4_case(batch, ctx, new, 8, 2, 64, bs, "bf16", factor=(0.5, 2.0))
    blocks = c["k_pool"].shape[0]
    rounds = blocks // 25 + 2
    c["table"][0, :25 * rounds] = c["table"][0, :25].repeat(rounds)
    c["kv_len"][0] = 400 * rounds
    assert 400 * rounds > blocks * bs
    check(c, "bf16", [2], window=window)


@pytest.mark.parametrize("batch", [2, 80])
@pytest.mark.parametrize("d,bs", [(64, 8), (128, 32), (256, 16)])
def test_blocks_behind_the_window_may_be_gone(batch, d, bs):
    """Their table entries name no block; the copy does not look at them either."""
    new = [1] * batch
    new[-1] = 150
    ctx = [90 + 7 * i % 300 for i in range(batch)]
    ctx[-1] = 1000
    c = fp4_case(d + batch, ctx, new, 4, 1, d, bs, "fp16")
    window = 150
    whole = host(c["table"]).copy()     # (the oracle looks every block up before it masks)
    for b in range(batch):
        gone = max(0, ctx[b] + 1 - window) // bs        # blocks of tokens that no row sees
        c["table"][b, :gone] = -1 if b % 2 else 1 << 24
    assert int(c["table"][-1, (1001 - window) // 128 * 128 // bs]) in (-1, 1 << 24)   # such tokens share the copy's first block
    check(c, "fp16", [batch - 1], window=window, table=whole)
