"""GPU parity of paged_attention against the float64 oracle: types, head
layouts, page sizes, lengths from zero and one token to several tiles, masks
that leave rows empty, NaN in every row that a request does not own."""

import numpy as np
import pytest

from oracle import paged_oracle
from tests.paged_cases import check_attention, host, paged_case

pytestmark = pytest.mark.gpu


def _run(sp, case, ref=True, lse=True, **kw):
    import torch
    q = case["q"]
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    ls = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda") if lse else None
    ws = sp.make_attention_workspace(q, case["kv_len"].numel(), case["k_pool"])
    sp.paged_attention(q, case["q_off"], case["kv_len"], case["table"], case["k_pool"], case["v_pool"], out=out,
                       lse=ls, ws=ws, **kw)
    assert sp.device_status(ws) == 0
    return out, ls


def _check(sp, ctx, new, hq, hk, d, bs, dtype, seed=0, q_gain=1.0, spare=3, **kw):
    case = paged_case(seed, ctx, new, hq, hk, d, bs, dtype, spare_rows=spare, q_gain=q_gain)
    out, lse = _run(sp, case, **kw)
    kv = host(case["kv_len"])
    ref = paged_oracle.paged_attention(host(case["q"]), host(case["q_off"]), kv, host(case["table"]),
                                       host(case["k_pool"]), host(case["v_pool"]), **kw)
    n = sum(new)
    check_attention(out, lse, ref, kv, d, dtype, n)
    # rows behind the last request stay as they were
    assert (host(out)[n:] == 7.0).all() and (host(lse)[n:] == 7.0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_single_tokens_over_ragged_contexts(cuda_lib, d, dtype):
    ctx = [0, 1, 7, 8, 126, 127, 128, 129, 255, 256, 700, 1500]
    _check(cuda_lib, ctx, [1] * len(ctx), 8, 2, d, 16, dtype, seed=d)


@pytest.mark.parametrize("d,bs", [(64, 8), (64, 256), (128, 32), (128, 128), (256, 16), (256, 64)])
def test_chunks_with_requests_of_no_and_one_token(cuda_lib, d, bs):
    ctx = [300, 5, 0, 0, 64, 1000]
    new = [130, 0, 1, 77, 64, 9]
    _check(cuda_lib, ctx, new, 4, 2, d, bs, "bf16", seed=bs)


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (10, 2), (7, 1), (6, 2), (16, 1), (48, 1), (128, 1), (5, 5)])
def test_groups_of_query_heads(cuda_lib, hq, hk):
    _check(cuda_lib, [100, 0, 33], [40, 150, 1], hq, hk, 64, 32, "bf16", seed=hq)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 500])
def test_sliding_window(cuda_lib, d, window):
    _check(cuda_lib, [400, 0, 1000, 129], [70, 300, 1, 130], 6, 2, d, 16, "fp16", seed=window, window=window)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_without_causality(cuda_lib, d):
    _check(cuda_lib, [90, 0, 257], [40, 128, 1], 4, 4, d, 64, "bf16", seed=d, causal=False)


@pytest.mark.parametrize("d", [64, 256])
def test_longer_contexts_split_over_many_ctas(cuda_lib, d):
    _check(cuda_lib, [9000, 200], [3, 1], 4, 1, d, 128, "bf16", seed=5)


@pytest.mark.parametrize("d,hq,hk", [(64, 6, 2), (128, 16, 4), (256, 8, 2)])
def test_last_keys_of_a_long_context_end_inside_a_tile(cuda_lib, d, hq, hk):
    """Many key tiles for each CTA, the last one partly behind the end."""
    _check(cuda_lib, [32768], [8], hq, hk, d, 16, "bf16", seed=12)
    _check(cuda_lib, [6001, 12000, 16383, 4097, 8200, 777], [1, 1, 1, 1, 3, 1], hq, hk, d, 16, "bf16", seed=13)


def test_prompt_of_several_query_tiles(cuda_lib):
    _check(cuda_lib, [0], [1100], 4, 1, 128, 64, "bf16", seed=9)
    _check(cuda_lib, [37], [700], 2, 1, 256, 16, "bf16", seed=10)
    _check(cuda_lib, [37], [901], 3, 1, 64, 16, "fp16", seed=11)
    _check(cuda_lib, [0], [2500], 8, 2, 256, 64, "bf16", seed=14)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_logits_move_the_running_maximum(cuda_lib, d):
    """Logits of up to some hundreds: the maximum moves in most tiles, by far
    more than any threshold, and most weights underflow."""
    _check(cuda_lib, [1200, 0], [5, 260], 4, 2, d, 32, "bf16", seed=d, q_gain=30.0)


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(cuda_lib, causal):
    """kv_len below the number of new tokens: the first tokens see nothing and
    give 0 and -inf; kv_len = 0 gives that for all."""
    import torch
    sp = cuda_lib
    case = paged_case(3, [0, 0, 10], [200, 30, 3], 4, 2, 128, 16, "bf16")
    case["kv_len"] = torch.tensor([150, 0, 13], dtype=torch.int32, device="cuda")
    out, lse = _run(sp, case, causal=causal)
    kv = host(case["kv_len"])
    ref = paged_oracle.paged_attention(host(case["q"]), host(case["q_off"]), kv, host(case["table"]),
                                       host(case["k_pool"]), host(case["v_pool"]), causal=causal)
    check_attention(out, lse, ref, kv, 128, "bf16", 233)
    assert np.isneginf(host(lse)[200:230]).all() and (host(out)[200:230] == 0).all()


def test_strided_queries_outputs_and_pools(cuda_lib):
    """q as a view of fused projections, out as a view of a wider tensor, pools
    whose heads and rows are views of wider rows."""
    import torch
    sp = cuda_lib
    hq, hk, d, bs = 6, 2, 64, 16
    case = paged_case(21, [50, 300], [20, 33], hq, hk, d, bs, "bf16")
    want, _ = _run(sp, case)
    n = case["q"].shape[0]
    fused = torch.randn(n, hq + 2 * hk, d, device="cuda").to(torch.bfloat16)
    fused[:, 1:1 + hq] = case["q"]
    wide = torch.zeros(n, hq, 2 * d, dtype=torch.bfloat16, device="cuda")
    nb = case["k_pool"].shape[0]
    both = torch.full((nb, bs, 2, hk, d + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    both[:, :, 0, :, :d] = case["k_pool"]
    both[:, :, 1, :, :d] = case["v_pool"]
    sp.paged_attention(fused[:, 1:1 + hq], case["q_off"], case["kv_len"], case["table"], both[:, :, 0, :, :d],
                       both[:, :, 1, :, :d], out=wide[:, :, d:])
    assert torch.equal(wide[:, :, d:], want)
    assert (wide[:, :, :d] == 0).all()


def test_bad_lengths_and_blocks_set_the_status(cuda_lib):
    import torch
    sp = cuda_lib
    case = paged_case(4, [40, 60], [3, 2], 4, 2, 64, 16, "bf16", poison=False)
    q = case["q"]

    def call(**kw):
        c = dict(case, **kw)
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        ws = sp.make_attention_workspace(q, 2, c["k_pool"])
        sp.paged_attention(q, c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"], out=out, ws=ws)
        return sp.device_status(ws), out

    def i32(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    assert call()[0] == 0
    for kw in (dict(q_off=i32(1, 3, 5)), dict(q_off=i32(0, 4, 3)), dict(q_off=i32(0, 3, 6)), dict(kv_len=i32(-1, 62)),
               dict(kv_len=i32(43, 100000))):
        status, out = call(**kw)
        assert status == 6 and (out == 7.0).all(), kw
    table = case["table"].clone()
    table[1, 2] = 1 << 20
    assert call(table=table)[0] == 6
    table[1, 2] = -3
    assert call(table=table)[0] == 6
    # an entry behind the request's last block is not read
    table = case["table"].clone()
    table[:, -1] = 1 << 30
    assert call(table=table)[0] == 0


def test_calls_on_streams_and_a_captured_call(cuda_lib):
    """Calls on three streams with workspaces of their own, a captured call
    replayed on new inputs, and two captured calls that share a workspace."""
    import torch
    sp = cuda_lib
    cases = [paged_case(30 + i, [700 * i, 10, 300], [60, 1, 5 + i], 8, 2, 128, 16, "bf16") for i in range(3)]
    want = [_run(sp, c)[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros_like(w) for w in want]
    wss = [sp.make_attention_workspace(c["q"], 3, c["k_pool"]) for c in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, st, o, ws in zip(cases, streams, outs, wss):
            sp.paged_attention(c["q"], c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"], out=o, ws=ws,
                               stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    ws = wss[0]
    graphs, goes = [], []
    for c in cases[:2]:
        o = torch.zeros_like(c["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sp.paged_attention(c["q"], c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"], out=o, ws=ws)
        graphs.append(g)
        goes.append(o)
    for _ in range(3):
        for g, o, w in zip(graphs, goes, want):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, w)
    # new lengths in place: fewer cached tokens of the first request
    c = cases[1]
    c["kv_len"][0] -= 100
    again, _ = _run(sp, c)
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(goes[1], again) and not torch.equal(again, want[1])


def test_repeated_calls_give_the_same_bits(cuda_lib):
    import torch
    sp = cuda_lib
    case = paged_case(50, [5000, 3, 900], [1, 300, 40], 16, 4, 128, 64, "bf16")
    a = _run(sp, case)
    for _ in range(5):
        b = _run(sp, case)
        n = 341
        assert torch.equal(a[0][:n], b[0][:n]) and torch.equal(a[1][:n], b[1][:n])


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("d,hq,hk,dtype", [(64, 4, 2, "fp16"), (128, 4, 1, "bf16"), (256, 2, 1, "bf16"), (128, 1, 1, "bf16")])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_row_masked_from_a_bad_value_is_not_touched_by_it(cuda_lib, d, hq, hk, dtype, value, window):
    """Infinity or NaN in two columns of one cached value, among the new tokens
    of a request with 400 of them: rows that see the token have no number in
    those columns, every other row and column is as without it. The same for a
    request long enough to be cut between CTAs."""
    import torch
    sp = cuda_lib
    ctx, new, bs = [30, 3000], [400, 130], 16
    case = paged_case(60 + d, ctx, new, hq, hk, d, bs, dtype)
    kv, table = host(case["kv_len"]), host(case["table"])
    bad = [30 + 211, 3000 + 57]   # cache indices
    cols = [3, d - 1]
    for b, j in enumerate(bad):
        case["v_pool"][int(table[b, j // bs]), j % bs][:, cols] = value
    # the oracle's result without the bad columns' contribution of those tokens
    clean = case["v_pool"].clone()
    for b, j in enumerate(bad):
        clean[int(table[b, j // bs]), j % bs][:, cols] = 0
    ref = paged_oracle.paged_attention(host(case["q"]), host(case["q_off"]), kv, table, host(case["k_pool"]),
                                       host(clean), window=window)
    out, lse = _run(sp, case, window=window)
    o = host(out)
    sees = np.zeros(o.shape[0], bool)
    for b, j in enumerate(bad):
        pos = kv[b] - new[b] + np.arange(new[b])
        lo = sum(new[:b])
        sees[lo:lo + new[b]] = (pos >= j) & ((window == 0) | (pos < j + window))
    assert sees.any() and not sees.all()
    assert not np.isfinite(o[sees][:, :, cols]).any()
    fixed = out.clone()
    mask = torch.zeros(o.shape, dtype=torch.bool)
    mask[torch.from_numpy(np.flatnonzero(sees))[:, None], :, torch.tensor(cols)] = True
    fixed[mask.cuda()] = torch.from_numpy(ref[0])[mask].to(fixed.dtype).cuda()
    check_attention(fixed, lse, ref, kv, d, dtype, sum(new))


def test_keys_that_are_no_numbers_reach_only_the_rows_that_see_them(cuda_lib):
    sp = cuda_lib
    case = paged_case(70, [10], [300], 4, 2, 128, 32, "bf16")
    table = host(case["table"])
    j = 10 + 140
    case["k_pool"][int(table[0, j // 32]), j % 32] = float("nan")
    out, lse = _run(sp, case)
    o = host(out)
    assert np.isfinite(o[:140]).all() and np.isnan(o[140:]).all() and np.isnan(host(lse)[140:]).all()


@pytest.mark.parametrize("bs,d", [(384, 128), (640, 64), (128, 256)])
def test_blocks_of_several_tiles(cuda_lib, bs, d):
    _check(cuda_lib, [1000, 3, 383], [5, 200, 2], 4, 2, d, bs, "bf16", seed=bs)


def test_batches_of_thousands_of_requests_and_of_many_query_tiles(cuda_lib):
    """More requests, and more query tiles, than a CTA lays out by itself."""
    rng = np.random.default_rng(3)
    new = (rng.random(3000) < 0.8).astype(int)
    _check(cuda_lib, rng.integers(0, 40, 3000).tolist(), new.tolist(), 4, 2, 64, 16, "bf16", seed=31)
    _check(cuda_lib, [5, 0, 90] * 150, [1, 3, 40] * 150, 8, 1, 128, 32, "fp16", seed=32)
    _check(cuda_lib, [0], [7000], 64, 1, 64, 64, "bf16", seed=33, window=100)


def test_no_new_tokens_and_no_cached_tokens(cuda_lib):
    sp = cuda_lib
    case = paged_case(5, [20, 0, 3], [0, 0, 0], 4, 2, 128, 16, "bf16", spare_rows=4)
    out, lse = _run(sp, case)
    assert (host(out) == 7.0).all() and (host(lse) == 7.0).all()


def test_outputs_aligned_to_16_bytes_only(cuda_lib):
    import torch
    sp = cuda_lib
    for d in (64, 128, 256):
        case = paged_case(40 + d, [50, 700], [130, 3], 4, 2, d, 16, "bf16")
        want, _ = _run(sp, case)
        wide = torch.zeros(133, 4, d + 8, dtype=torch.bfloat16, device="cuda")
        sp.paged_attention(case["q"], case["q_off"], case["kv_len"], case["table"], case["k_pool"], case["v_pool"],
                           out=wide[:, :, 8:])
        assert torch.equal(wide[:, :, 8:], want) and (wide[:, :, :8] == 0).all()


def test_cache_rows_past_32_bit_offsets(cuda_lib):
    """Pools of 2^31 elements and more, with the request's blocks at both ends;
    the new tokens are stored there by append_kv."""
    import torch
    sp = cuda_lib
    hk, d, bs = 8, 256, 64
    blocks = 2 ** 31 // (hk * d * bs) + 40
    assert blocks * bs * hk * d > 2 ** 31
    pools = [torch.zeros(blocks, bs, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ids = [blocks - 1, 0, blocks - 2, 1, blocks - 3]
    n = 5 * bs - 7
    rng = np.random.default_rng(9)
    kv = [torch.from_numpy(rng.standard_normal((n, hk, d), dtype=np.float32)).cuda().bfloat16() for _ in range(2)]
    slots = (np.asarray(ids)[:, None] * bs + np.arange(bs)).reshape(-1)[:n].astype(np.int32)
    sp.append_kv(*kv, torch.from_numpy(slots).cuda(), *pools)
    q = torch.from_numpy(rng.standard_normal((3, hk, d), dtype=np.float32)).cuda().bfloat16()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lse = torch.zeros(3, hk, device="cuda")
    ws = sp.make_attention_workspace(q, 1, pools[0])
    out = sp.paged_attention(q, i32(0, 3), i32(n), i32(*ids)[None], *pools, lse=lse, ws=ws)
    assert sp.device_status(ws) == 0
    small = [host(p[torch.tensor(ids, device="cuda")]) for p in pools]
    ref = paged_oracle.paged_attention(host(q), [0, 3], [n], np.arange(5)[None], *small)
    check_attention(out, lse, ref, [n], d, "bf16", 3)


def test_waits_that_give_up_set_the_status_and_leave_the_workspace_usable(cuda_lib):
    """With one poll for every wait the first one that has to wait gives up;
    the call ends with SP_ERR_TIMEOUT and the next one is right."""
    import torch
    sp = cuda_lib
    for d in (64, 128, 256):
        case = paged_case(80 + d, [3000, 100], [1, 200], 4, 2, d, 16, "bf16")
        want, _ = _run(sp, case)
        ws = sp.make_attention_workspace(case["q"], 2, case["k_pool"])
        out = torch.zeros_like(case["q"])
        args = (case["q"], case["q_off"], case["kv_len"], case["table"], case["k_pool"], case["v_pool"])
        sp.paged_attention(*args, out=out, ws=ws, spin_limit=1)
        assert sp.device_status(ws) == 5
        sp.paged_attention(*args, out=out, ws=ws)
        assert sp.device_status(ws) == 0 and torch.equal(out, want)


def test_windows_longer_than_any_context_hide_nothing(cuda_lib):
    import torch
    sp = cuda_lib
    case = paged_case(90, [2000, 0], [130, 60], 4, 2, 128, 32, "bf16")
    want = _run(sp, case)
    for window in (2131, 1 << 30, (1 << 30) + 1, 2 ** 31 - 1):
        got = _run(sp, case, window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), window


def test_blocks_shared_by_requests(cuda_lib):
    """Two requests whose tables name the same blocks for their common start."""
    import torch
    sp = cuda_lib
    bs, d = 16, 64
    case = paged_case(91, [64, 64], [5, 9], 4, 2, d, bs, "bf16")
    case["table"][1, :4] = case["table"][0, :4]
    out, lse = _run(sp, case)
    kv = host(case["kv_len"])
    ref = paged_oracle.paged_attention(host(case["q"]), host(case["q_off"]), kv, host(case["table"]),
                                       host(case["k_pool"]), host(case["v_pool"]))
    check_attention(out, lse, ref, kv, d, "bf16", 14)
    assert torch.isfinite(out.float()).all()
