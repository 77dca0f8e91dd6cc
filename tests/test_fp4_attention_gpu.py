"""Attention over the 4-bit cache against the float64 oracle on the values that
the pools stand for."""

import numpy as np
import pytest

from oracle import paged_oracle
from tests.fp4_cases import check_attention, dev, fp4_case
from tests.paged_cases import host

pytestmark = pytest.mark.gpu


def attend(c, causal=True, window=0, scale=0.0, max_new=None, kv_tokens=None, spare=None, ws=None, **more):
    import torch

    import speculative_prefill_token_gb300 as sp
    if ws is None:
        ws = sp.make_attention_fp4_workspace(c["q"], c["kv_len"].numel(), c["k_pool"], max_new=max_new, kv_tokens=kv_tokens)
    out = torch.full_like(c["q"], 7.0)
    lse = torch.full(c["q"].shape[:2], 7.0, dtype=torch.float32, device="cuda")
    sp.paged_attention_fp4(c["q"], c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"], causal=causal,
                           window=window, scale=scale, k_scale=c["k_scale"], v_scale=c["v_scale"], out=out, lse=lse,
                           max_new=max_new, ws=ws, **more)
    return out, lse, sp.device_status(ws)


def reference(c, causal=True, window=0, scale=0.0):
    return paged_oracle.paged_attention(host(c["q"]), host(c["q_off"]), host(c["kv_len"]), host(c["table"]),
                                        np.nan_to_num(c["k"]), np.nan_to_num(c["v"]), causal, window, scale or None)


def check(c, dtype, causal=True, window=0, scale=0.0, **more):
    out, lse, status = attend(c, causal, window, scale, **more)
    assert status == 0
    tokens = int(c["q_off"][-1])
    d = c["q"].shape[2]
    check_attention(out, lse, reference(c, causal, window, scale), host(c["kv_len"]), d, dtype, tokens,
                    float(np.nanmax(np.abs(c["v"]))))
    # rows behind the last request stay as they were
    assert (out[tokens:] == 7.0).all() and (lse[tokens:] == 7.0).all()
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hk", [(4, 2), (5, 1), (8, 1), (3, 3), (24, 2)])
def test_decode_steps(dtype, d, hq, hk):
    ctx = [0, 1, 7, 62, 63, 64, 127, 200, 511, 1000]
    c = fp4_case(d + hq, ctx, [1] * len(ctx), hq, hk, d, 16, dtype, spare_rows=3, factor=(0.5, 0.07))
    check(c, dtype, max_new=1)


@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128, 384])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_block_sizes(bs, d):
    c = fp4_case(bs + d, [300, 0, 999, 64], [1, 3, 40, 1], 6, 2, d, bs, "bf16")
    check(c, "bf16", kv_tokens=0)
    check(c, "bf16", window=70, kv_tokens=0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 33), (True, 5000)])
@pytest.mark.parametrize("kv_tokens", [0, None])
def test_mixed_lengths_and_masks(dtype, causal, window, kv_tokens):
    c = fp4_case(5, [0, 0, 90, 700, 1, 333, 64], [1, 130, 0, 1, 63, 300, 64], 10, 2, 128, 32, dtype, spare_rows=5,
                 factor=(1.0, 2.0))
    check(c, dtype, causal, window, kv_tokens=kv_tokens)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kv_tokens", [0, None])
def test_long_contexts_are_cut_between_ctas(d, kv_tokens):
    c = fp4_case(d, [30011, 0, 12345], [8, 1, 1], 8, 2, d, 64, "bf16")
    check(c, "bf16", max_new=8, kv_tokens=kv_tokens)
    check(c, "bf16", window=20000, max_new=8, kv_tokens=kv_tokens)


@pytest.mark.parametrize("kv_tokens", [0, None, 600])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts_and_chunks(d, kv_tokens):
    """Requests with many rows; where 600 cached tokens fit into the workspace's
    copy, one request is read through it and the others are not."""
    c = fp4_case(d, [0, 100, 0, 512], [500, 450, 1, 129], 8, 2, d, 64, "bf16", spare_rows=1, factor=(0.3, 1.0))
    check(c, "bf16", kv_tokens=kv_tokens)


def test_more_new_tokens_than_cached():
    c = fp4_case(1, [0, 0], [40, 5], 4, 2, 64, 16, "bf16")
    c["kv_len"] = dev(np.array([11, 0], dtype=np.int32))
    for kv_tokens in (0, None):
        out, lse, status = attend(c, kv_tokens=kv_tokens)
        assert status == 0
        ref = reference(c)
        check_attention(out, lse, ref, [11], 64, "bf16", 45, 6.0 * 448)
        assert (host(out)[:29] == 0).all() and np.isneginf(host(lse)[:29]).all()
        assert (host(out)[40:] == 0).all() and np.isneginf(host(lse)[40:]).all()


def test_large_logits_and_sinks():
    """A key that outweighs all others early, and logits that climb along the context."""
    c = fp4_case(3, [4000], [2], 4, 1, 128, 64, "bf16", q_gain=30.0)
    check(c, "bf16")


@pytest.mark.parametrize("batch", [65, 200, 1100, 3000])
def test_many_requests(batch):
    rng = np.random.default_rng(batch)
    ctx = rng.integers(0, 60, batch).tolist()
    new = rng.integers(0, 2, batch).tolist()
    c = fp4_case(batch, ctx, new, 4, 2, 64, 8, "bf16")
    check(c, "bf16", max_new=1)


@pytest.mark.parametrize("kv_tokens", [0, None])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_values_that_are_no_number_reach_only_rows_that_see_them(d, kv_tokens):
    """NaN scales in a key and in a value of the new tokens."""
    hq, hk, bs, ctx, new = 6, 2, 32, 100, 40
    c = fp4_case(9, [ctx], [new], hq, hk, d, bs, "bf16")
    width = c["table"].shape[1]
    at = lambda j: (int(c["table"][0, j // bs]), j % bs)  # noqa: E731
    assert width > 4
    for pool, name, j, head, group in ((c["k_pool"], "k", ctx + 20, 0, 1), (c["v_pool"], "v", ctx + 30, 1, d // 16 - 1)):
        blk, row = at(j)
        pool[blk, head, row // 8, 4 * d + row % 8 * (d // 16) + group] = 127
    out, lse, status = attend(c, kv_tokens=kv_tokens)
    assert status == 0
    ref = reference(c)
    from tests.fp4_cases import attention_bounds
    tol_out, tol_lse = attention_bounds(ref, [ctx + new], d, "bf16", 6.0)
    o, s = host(out), host(lse)
    bad = np.zeros(o.shape, dtype=bool)
    bad[20:, :hq // hk] = True                         # a key of KV head 0: every element
    bad[30:, hq // hk:, d - 16:] = True                # a value of KV head 1: the last group
    assert np.isnan(o[bad]).all()
    assert (np.abs(o - ref[0]) <= tol_out)[~bad].all()
    assert np.isnan(s[20:, :hq // hk]).all()
    assert (np.abs(s - ref[1]) <= tol_lse)[:20].all() and (np.abs(s - ref[1]) <= tol_lse)[:, hq // hk:].all()


def test_queries_that_are_no_number_stay_in_their_row():
    import torch
    c = fp4_case(4, [150], [3], 6, 2, 128, 16, "bf16")
    c["q"][1, 2, 5] = float("nan")
    c["q"][2, 0, 7] = float("inf")
    out, lse, status = attend(c)
    good = torch.ones(3, 6, dtype=torch.bool)
    good[1, 2] = good[2, 0] = False
    q = c["q"].clone()
    q[1, 2] = q[2, 0] = 0
    ref = reference(dict(c, q=q))
    from tests.fp4_cases import attention_bounds
    tol, _ = attention_bounds(ref, [153], 128, "bf16", 6.0)
    assert (np.abs(host(out) - ref[0]) <= tol)[good.numpy()].all()
    assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[1, 2])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_tiny_and_huge_queries(dtype):
    """Rows far from one, within the type: their scaling is exact."""
    c = fp4_case(6, [90, 90], [1, 1], 4, 2, 64, 16, dtype)
    c["q"][0] *= 2.0 ** -13
    c["q"][1] *= 2.0 ** 9
    check(c, dtype)
    if dtype == "bf16":
        c["q"][0] *= 2.0 ** -90
        check(c, dtype)
        check(c, dtype, scale=2.0 ** 80)
        c["q"][1] *= 2.0 ** 100
        check(c, dtype, scale=2.0 ** -110)


def test_strided_queries_outputs_and_pools():
    import torch

    import speculative_prefill_token_gb300 as sp
    c = fp4_case(8, [77, 300], [2, 1], 6, 2, 64, 16, "bf16")
    t, hq, d = c["q"].shape
    wide = torch.zeros(t, hq + 4, d, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + hq] = c["q"]
    heads_first = torch.full((hq, t, d), 7.0, dtype=torch.bfloat16, device="cuda")
    # two layers' pools interleaved by block
    both = [torch.randint(0, 255, (p.shape[0], 2, *p.shape[1:]), dtype=torch.uint8, device="cuda") for p in (c["k_pool"], c["v_pool"])]
    for w, p in zip(both, (c["k_pool"], c["v_pool"])):
        w[:, 1] = p
    out = sp.paged_attention_fp4(wide[:, 2:2 + hq], c["q_off"], c["kv_len"], c["table"], both[0][:, 1], both[1][:, 1],
                                 out=heads_first.transpose(0, 1))
    want, _, _ = attend(c)
    assert torch.equal(out, want)


def test_results_do_not_depend_on_timing_or_neighbours():
    import torch
    c = fp4_case(11, [20000, 5, 0, 300], [1, 1, 200, 7], 8, 2, 128, 64, "bf16")
    a = attend(c)
    for _ in range(3):
        b = attend(c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_errors_on_the_device():
    for change in (dict(q_off=[1, 2, 3]), dict(q_off=[0, 2, 1]), dict(q_off=[0, 1, 9]), dict(kv_len=[10, -1]),
                   dict(kv_len=[10, 100000])):
        c = fp4_case(12, [30, 30], [1, 2], 4, 2, 64, 16, "bf16")
        for k, v in change.items():
            c[k] = dev(np.array(v, dtype=np.int32))
        for kv_tokens in (0, None):
            out, lse, status = attend(c, kv_tokens=kv_tokens)
            assert status == 6, change
            assert (out == 7.0).all() and (lse == 7.0).all()
    # more new tokens than max_new
    c = fp4_case(12, [30, 30], [1, 2], 4, 2, 64, 16, "bf16")
    assert attend(c, max_new=1)[2] == 6
    # a block id outside the pool reads block 0
    c["table"][0, 0] = 1 << 20
    out, _, status = attend(c)
    assert status == 6
    c["table"][0, 0] = 0
    want, _, status = attend(c)
    assert status == 0
    assert out[1:].equal(want[1:])


def test_a_wait_that_gives_up():
    """A limit of one poll, in the attention over the 16-bit copy: the call
    returns with a status, and the next one works."""
    import speculative_prefill_token_gb300 as sp
    c = fp4_case(13, [3000], [40], 4, 2, 128, 64, "bf16")
    ws = sp.make_attention_fp4_workspace(c["q"], 1, c["k_pool"])
    seen = {attend(c, ws=ws, spin_limit=1)[2] for _ in range(8)}
    assert seen <= {0, 5} and 5 in seen
    check(c, "bf16", ws=ws)


def test_captured_steps_share_a_workspace_and_see_new_lengths():
    import torch

    import speculative_prefill_token_gb300 as sp
    c = fp4_case(14, [400, 31], [1, 1], 4, 2, 128, 16, "bf16")
    ws = sp.make_attention_fp4_workspace(c["q"], 2, c["k_pool"], max_new=1)
    outs = [torch.zeros_like(c["q"]) for _ in range(2)]
    q2 = c["q"] * 0.5

    def step(q, out):
        sp.paged_attention_fp4(q, c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"], out=out, max_new=1, ws=ws)

    step(c["q"], outs[0])
    torch.cuda.synchronize()
    graphs = []
    for q, out in zip((c["q"], q2), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(q, out)
        graphs.append(g)
    for kv in ([401, 32], [17, 1], [300, 20]):
        c["kv_len"].copy_(dev(np.array(kv, dtype=np.int32)))
        for g in graphs:
            g.replay()
        for q, out in zip((c["q"], q2), outs):
            got = out.clone()
            assert torch.equal(got, attend(dict(c, q=q), max_new=1)[0])
    assert sp.device_status(ws) == 0


def test_another_stream():
    import torch
    c = fp4_case(15, [1000, 3], [1, 1], 8, 2, 128, 64, "bf16")
    want = attend(c)[0]
    st = torch.cuda.Stream()
    import speculative_prefill_token_gb300 as sp
    st.wait_stream(torch.cuda.current_stream())
    out = sp.paged_attention_fp4(c["q"], c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"], stream=st)
    st.synchronize()
    assert torch.equal(out, want)
