"""Requests of the 4-bit attention that are read through the 16-bit copy in the
workspace. Every test looks for a row of the cache in the workspace, so that it
fails when its request no longer goes that way."""

import numpy as np
import pytest

from oracle import paged_oracle
from tests.fp4_cases import attention_bounds, check_attention, dev, fp4_case
from tests.paged_cases import host
from tests.test_fp4_rows_gpu import bound_of_fp16_weights

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


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 33), (True, 5000)])
@pytest.mark.parametrize("batch", [5, 90])
def test_masks(dtype, causal, window, batch):
    """Layouts of the copy by a warp and by a block; a chunk of 190 rows is too short for it."""
    import speculative_prefill_token_gb300 as sp
    new, ctx = [1] * batch, [3 + 11 * i % 400 for i in range(batch)]
    new[1], new[2], new[batch - 2] = 60, 38, 170
    ctx[1], ctx[batch - 2] = 0, 777
    c = fp4_case(batch, ctx, new, 5, 1, 64, 32, dtype, spare_rows=2, factor=(0.25, 3.0))
    ws = sp.make_attention_fp4_workspace(c["q"], batch, c["k_pool"])
    check(c, dtype, [1, batch - 2], causal, window, ws=ws)
    assert not held_in_16_bits(c, ws, 2, ctx[2] + 37)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("factor", [(1.0, 1.0), (0.5, 3.0)])
def test_values_that_are_no_number_reach_only_rows_that_see_them(d, factor):
    """NaN scales in a key and in a value of the new tokens: rows that are taken one by one, the pool's factor in them."""
    hq, hk, bs, ctx, new = 6, 2, 32, 100, 100
    c = fp4_case(9, [ctx], [new], hq, hk, d, bs, "bf16", factor=factor)
    at = lambda j: (int(c["table"][0, j // bs]), j % bs)  # noqa: E731
    for pool, j, head, group in ((c["k_pool"], ctx + 20, 0, 1), (c["v_pool"], ctx + 30, 1, d // 16 - 1)):
        blk, row = at(j)
        pool[blk, head, row // 8, 4 * d + row % 8 * (d // 16) + group] = 127
    out, lse, status = attend(c, [0])
    assert status == 0
    ref = paged_oracle.paged_attention(host(c["q"]), host(c["q_off"]), host(c["kv_len"]), host(c["table"]),
                                       np.nan_to_num(c["k"]), np.nan_to_num(c["v"]))
    tol_out, tol_lse = attention_bounds(ref, [ctx + new], d, "bf16", float(np.nanmax(np.abs(c["v"]))))
    o, s = host(out), host(lse)
    bad = np.zeros(o.shape, dtype=bool)
    bad[20:, :hq // hk] = True                         # a key of KV head 0: every element
    bad[30:, hq // hk:, d - 16:] = True                # a value of KV head 1: the last group
    assert np.isnan(o[bad]).all()
    assert (np.abs(o - ref[0]) <= tol_out)[~bad].all()
    assert np.isnan(s[20:, :hq // hk]).all()
    assert (np.abs(s - ref[1]) <= tol_lse)[:20].all() and (np.abs(s - ref[1]) <= tol_lse)[:, hq // hk:].all()


def test_more_new_tokens_than_cached():
    c = fp4_case(1, [0, 0], [200, 5], 4, 2, 64, 16, "bf16", factor=(1.0, 0.5))
    c["kv_len"] = dev(np.array([60, 0], dtype=np.int32))
    out, lse, status = attend(c, [0])
    assert status == 0
    ref = paged_oracle.paged_attention(host(c["q"]), host(c["q_off"]), host(c["kv_len"]), host(c["table"]),
                                       np.nan_to_num(c["k"]), np.nan_to_num(c["v"]))
    check_attention(out, lse, ref, [60], 64, "bf16", 205, 6.0)
    for x in (slice(0, 140), slice(200, 205)):
        assert (host(out)[x] == 0).all() and np.isneginf(host(lse)[x]).all()


def test_a_wait_that_gives_up():
    """A limit of one poll in the attention over the copy: the call returns with a status, and the next one works."""
    import speculative_prefill_token_gb300 as sp
    c = fp4_case(13, [3000], [200], 4, 2, 128, 64, "bf16")
    ws = sp.make_attention_fp4_workspace(c["q"], 1, c["k_pool"])
    seen = {attend(c, [0], ws=ws, spin_limit=1)[2] for _ in range(8)}
    assert seen <= {0, 5} and 5 in seen
    check(c, "bf16", [0], ws=ws)


def test_captured_chunks_and_steps_share_a_workspace():
    """Two graphs, one with a chunk through the copy and one of decode steps, replayed in turn with other lengths."""
    import torch

    import speculative_prefill_token_gb300 as sp
    chunk = fp4_case(21, [900, 40], [120, 1], 4, 1, 128, 16, "bf16")
    steps = dict(chunk, q=chunk["q"][:2].clone(), q_off=dev(np.array([0, 1, 2], dtype=np.int32)))
    ws = sp.make_attention_fp4_workspace(chunk["q"], 2, chunk["k_pool"])
    cases, outs, graphs = [chunk, steps], [], []
    kv = chunk["kv_len"].clone()
    for c in cases:
        outs.append(torch.zeros_like(c["q"]))
        run = lambda: sp.paged_attention_fp4(c["q"], c["q_off"], kv, c["table"], c["k_pool"], c["v_pool"], window=300,  # noqa: E731
                                             out=outs[-1], ws=ws)
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append(graph)
    for lengths in ([1020, 41], [700, 3], [121, 30]):
        kv.copy_(dev(np.array(lengths, dtype=np.int32)))
        for g in graphs + graphs[::-1]:
            g.replay()
        for c, out in zip(cases, outs):
            assert torch.equal(out, attend(dict(c, kv_len=kv), window=300)[0])
    assert sp.device_status(ws) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_weights_have_11_bits(d):
    """As they have on the 4-bit rows: a bf16 chunk's error does not depend on the way it goes."""
    c = fp4_case(d, [3000, 0, 1], [150, 140, 1], 8, 2, d, 32, "bf16", factor=(0.5, 2.0))
    ref = paged_oracle.paged_attention(host(c["q"]), host(c["q_off"]), host(c["kv_len"]), host(c["table"]),
                                       np.nan_to_num(c["k"]), np.nan_to_num(c["v"]))
    out, _, status = attend(c, [0, 1])
    assert status == 0
    assert (np.abs(host(out) - ref[0]) <= bound_of_fp16_weights(c, ref)).all()
