"""The operators as they are used together: prompts scored, their kept tokens
stored in 4 bits, decoded, forked, compacted and freed, with the lengths on the
device."""

import numpy as np
import pytest

from oracle import fp4_oracle, paged_oracle
from synth import get_workload, make_inputs
from tests.fp4_cases import check_attention, dev
from tests.gpu_helpers import to_device
from tests.paged_cases import host

pytestmark = pytest.mark.gpu


def i32(*v):
    return dev(np.array(v, dtype=np.int32))


@pytest.mark.parametrize("captured", [False, True])
def test_score_store_decode_fork_and_free(cuda_lib, captured):
    import torch
    sp = cuda_lib
    w = get_workload("tiny")
    q, k, off = to_device(make_inputs(w))
    out = sp.specprefill_score(q, k, off, sp.SelectionParams(**w.selection_kwargs()))
    n = int(out.n_kept)
    bs, hq, hk, d, cap, rows = 16, 8, 2, 128, w.lengths[0], 4
    blocks = 3 * (cap // bs) + 8
    gen = torch.Generator(device="cuda").manual_seed(0)
    pools = [sp.make_pool_fp4(blocks, bs, hk, d) for _ in range(2)]
    table = torch.full((rows, cap // bs + 2), -1, dtype=torch.int32, device="cuda")
    free, shared = torch.arange(blocks, dtype=torch.int32, device="cuda"), torch.zeros(blocks, dtype=torch.int32, device="cuda")
    ctx, n_free, status = i32(0, 0, 0, 0), i32(blocks), i32(0)
    angle = torch.arange(cap + 8, device="cuda")[:, None] * 1e4 ** (-torch.arange(d // 2, device="cuda") * 2.0 / d)
    turn = torch.cat([angle.cos(), angle.sin()], 1).contiguous()
    # the kept tokens of the prompt, request 0 (the others have none)
    qkv = torch.randn(cap, hq + 2 * hk, d, device="cuda", generator=gen).bfloat16()
    new_off = torch.cat([out.kept_off, out.kept_off[-1:].expand(rows - 1)]).contiguous()
    slots, kv, left = sp.block_tables(ctx, new_off, free, n_free, table, bs, n_tokens=cap, status=status)
    qr = sp.append_kv_fp4(qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, *pools, q=qkv[:, :hq], positions=out.kept_pos,
                          cos_sin=turn, n_new=out.n_kept, k_scale=0.5, v_scale=0.25, status=status)
    ws = sp.make_attention_fp4_workspace(qr, rows, pools[0])
    o = sp.paged_attention_fp4(qr, new_off, kv, table, *pools, k_scale=0.5, v_scale=0.25, ws=ws)

    def reference(q, off, kv):
        k, v = (fp4_oracle.values(host(p), f) for p, f in zip(pools, (0.5, 0.25)))
        return paged_oracle.paged_attention(host(q), host(off), host(kv), host(table), np.nan_to_num(k), np.nan_to_num(v))

    check_attention(o, None, reference(qr, new_off, kv), host(kv), d, "bf16", n, 30.0)
    # the keys are what the definition makes of the rotated rows
    codes, scales = fp4_oracle.encode(fp4_oracle.rotate32(host(qkv[:n, hq:hq + hk]).astype(np.float32), host(out.kept_pos)[:n],
                                                          host(turn).astype(np.float32)), 0.5)
    at = host(slots)[:n]
    got = fp4_oracle.unpack(host(pools[0]))
    assert np.array_equal(got[0][at // bs, at % bs], codes) and np.array_equal(got[1][at // bs, at % bs], scales)
    # three continuations
    kv, cs, cd, left = sp.fork_blocks(i32(0, 0, 0), i32(2, 1, 3), kv, table, shared, free, left, bs, status=status)
    sp.copy_kv(pools, cs, cd, rows=bs, status=status)
    assert int(status) == 0 and host(kv).tolist() == [n] * 4
    # decode steps of all four, each with tokens of its own
    one = i32(0, 1, 2, 3, 4)
    s = dict(ctx=kv.clone(), n_free=left.clone(), slots=i32(0, 0, 0, 0), kv=i32(0, 0, 0, 0), left=i32(0),
             qkv=torch.zeros(rows, hq + 2 * hk, d, dtype=torch.bfloat16, device="cuda"), pos=i32(0, 0, 0, 0))
    outs = dict(q=torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda"),
                o=torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda"))
    ws1 = sp.make_attention_fp4_workspace(outs["q"], rows, pools[0], max_new=1)

    def step():
        sp.block_tables(s["ctx"], one, free, s["n_free"], table, bs, slot_map=s["slots"], kv_len=s["kv"], n_left=s["left"],
                        status=status)
        sp.append_kv_fp4(s["qkv"][:, hq:hq + hk], s["qkv"][:, hq + hk:], s["slots"], *pools, q=s["qkv"][:, :hq],
                         q_out=outs["q"], positions=s["pos"], cos_sin=turn, k_scale=0.5, v_scale=0.25, status=status)
        sp.paged_attention_fp4(outs["q"], one, s["kv"], table, *pools, k_scale=0.5, v_scale=0.25, out=outs["o"], max_new=1, ws=ws1)
        s["ctx"].copy_(torch.where(status == 0, s["kv"], s["ctx"]))
        s["n_free"].copy_(torch.where(status == 0, s["left"], s["n_free"]))

    run = step
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay
    for i in range(20):
        s["qkv"].copy_(torch.randn(rows, hq + 2 * hk, d, device="cuda", generator=gen).bfloat16())
        s["pos"].fill_(cap - 20 + i)
        run()
        check_attention(outs["o"], None, reference(outs["q"], one, s["kv"]), host(s["kv"]), d, "bf16", rows, 30.0)
    assert int(status) == 0 and sp.device_status(ws1) == 0 and host(s["ctx"]).tolist() == [n + 20] * 4
    # every second cached token of request 1 moves to blocks of its own, in 4 bits; the old row is freed
    keep = torch.arange(0, n + 20, 2, dtype=torch.int32, device="cuda")
    m = keep.numel()
    table2 = torch.full((1, table.shape[1]), -1, dtype=torch.int32, device="cuda")
    slots2, kv2, left = sp.block_tables(i32(0), i32(0, m), free, s["n_free"], table2, bs, n_tokens=m, status=status)
    sp.copy_kv(pools, keep, slots2, block_table=table[1:2], src_off=i32(0, m), status=status)
    both = host(sp.unpack_fp4(pools[1], slots=slots2))
    row = host(table)[1]
    old = (row[host(keep) // bs] * bs + host(keep) % bs).astype(np.int32)
    assert np.array_equal(both, host(sp.unpack_fp4(pools[1], slots=dev(old))))
    ctx2, left = sp.free_blocks(s["ctx"], i32(n + 20, 0, n + 20, 0), table, shared, free, left, bs, status=status)
    ctx2, left = sp.free_blocks(ctx2, i32(0, 0, 0, 0), table, shared, free, left, bs, status=status)
    ctx2, left = sp.free_blocks(kv2, i32(0), table2, shared, free, left, bs, status=status)
    assert int(status) == 0 and int(left) == blocks and not shared.any()
    assert sorted(host(free).tolist()) == list(range(blocks))


def test_scoring_over_keys_read_back(cuda_lib):
    """A draft's cache in 4 bits: its keys read back are scored like any 16-bit cache."""
    import torch
    sp = cuda_lib
    w = get_workload("tiny")
    q, k, off = to_device(make_inputs(w))
    bs, n = 16, w.lengths[0]
    hk, d = w.n_kv_heads, w.head_dim
    p = sp.SelectionParams(**w.selection_kwargs())
    table = torch.randperm(n // bs, device="cuda").to(torch.int32)[None].contiguous()
    slot = (table[0].long().repeat_interleave(bs) * bs + torch.arange(bs, device="cuda").repeat(n // bs)).to(torch.int32)
    layers, dense = [], []
    for layer in range(k.shape[0]):
        pools = [sp.make_pool_fp4(n // bs, bs, hk, d) for _ in range(2)]
        rows = k[layer].view(torch.bfloat16)
        sp.append_kv_fp4(rows, rows, slot, *pools)
        layers.append(sp.unpack_fp4(pools[0]))
        dense.append(sp.unpack_fp4(pools[0], slots=slot))
    a = sp.specprefill_score_kv(q, layers, off, n, p, block_table=table)
    b = sp.specprefill_score(q, torch.stack(dense).view(torch.int16), off, p)
    assert torch.equal(a.imp, b.imp) and int(a.n_kept) == int(b.n_kept)


def test_calls_on_two_streams(cuda_lib):
    """Two steps at once, a workspace each."""
    import torch
    from tests.fp4_cases import fp4_case
    sp = cuda_lib
    cases = [fp4_case(i, [5000 + i, 40], [1, 1], 8, 2, 128, 16, "bf16") for i in range(2)]
    args = [(c["q"], c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"]) for c in cases]
    want = [sp.paged_attention_fp4(*a) for a in args]
    ws = [sp.make_attention_fp4_workspace(c["q"], 2, c["k_pool"]) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(sp.paged_attention_fp4(*args[i], ws=ws[i], stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])


def test_a_small_workspace_is_refused(cuda_lib):
    from tests.fp4_cases import fp4_case
    sp = cuda_lib
    c = fp4_case(3, [50], [300], 8, 2, 64, 16, "bf16")
    ws = sp.make_attention_fp4_workspace(c["q"], 1, c["k_pool"], max_new=1)
    with pytest.raises(sp.SpecPrefillError):
        sp.paged_attention_fp4(c["q"], c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"], ws=ws)
    with pytest.raises(ValueError):
        sp.paged_attention_fp4(c["q"], c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"][:, :1], ws=ws)
    with pytest.raises(ValueError):
        sp.paged_attention_fp4(c["q"], c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"], max_new=0, ws=ws)


@pytest.mark.parametrize("fault", ["max_new", "kv_len", "q_off"])
def test_a_length_out_of_range_stops_the_chunks_of_the_others(cuda_lib, fault):
    """Nothing is written, by the kernels over 16 bits neither."""
    import torch
    from tests.fp4_cases import fp4_case
    sp = cuda_lib
    c = fp4_case(5, [500, 0, 90], [200, 130, 1], 8, 2, 128, 16, "bf16")
    off, kv = c["q_off"].clone(), c["kv_len"].clone()
    ws = sp.make_attention_fp4_workspace(c["q"], 3, c["k_pool"], kv_tokens=3000)
    args = dict(k_scale=1.0, v_scale=1.0, ws=ws)
    want = sp.paged_attention_fp4(c["q"], off, kv, c["table"], c["k_pool"], c["v_pool"], **args)
    assert sp.device_status(ws) == 0
    if fault == "max_new":
        ws = sp.make_attention_fp4_workspace(c["q"], 3, c["k_pool"], max_new=150, kv_tokens=3000)
        args.update(ws=ws, max_new=150)
    elif fault == "kv_len":
        kv[2] = 16 * c["table"].shape[1] + 1
    else:
        off[3] = off[2] - 1
    out = torch.full_like(want, 7.0)
    sp.paged_attention_fp4(c["q"], off, kv, c["table"], c["k_pool"], c["v_pool"], out=out, **args)
    assert sp.device_status(ws) == 6 and (out == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,hq,d,rot", [(1300, 32, 128, 128), (5001, 8, 64, 48), (700, 33, 256, 64)])
def test_many_rows_in_place(cuda_lib, dtype, n, hq, d, rot):
    """Queries that go in a launch of their own, in place, some rows not in use."""
    import torch
    from tests.paged_cases import torch_dtype
    sp = cuda_lib
    hk, bs, used = 2, 16, n - 3
    gen = torch.Generator(device="cuda").manual_seed(n)
    qkv = torch.randn(n, hq + 2 * hk, d, device="cuda", generator=gen).to(torch_dtype(dtype))
    turn = torch.randn(64, rot, device="cuda", generator=gen)
    pos = torch.randint(0, 64, (n,), device="cuda", generator=gen, dtype=torch.int32)
    blocks = -(-n // bs) + 1
    slots = torch.randperm(blocks * bs, device="cuda", generator=gen)[:n].to(torch.int32)
    slots[5] = -1
    pools = [sp.make_pool_fp4(blocks, bs, hk, d) for _ in range(2)]
    ref = [torch.zeros(blocks, bs, hk, d, dtype=torch_dtype(dtype), device="cuda") for _ in range(2)]
    want = sp.append_kv(qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, *ref, q=qkv[:, :hq], positions=pos, cos_sin=turn)
    before, status = qkv.clone(), i32(0)
    sp.append_kv_fp4(qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, *pools, q=qkv[:, :hq], q_out=qkv[:, :hq], positions=pos,
                     cos_sin=turn, n_new=i32(used), k_scale=0.5, status=status)
    assert int(status) == 0
    assert torch.equal(qkv[:used, :hq], want[:used]) and torch.equal(qkv[used:], before[used:])
    assert torch.equal(qkv[:, hq:], before[:, hq:])
    x = host(before)
    rows = [fp4_oracle.rotate32(x[:, hq:hq + hk].astype(np.float32), host(pos), host(turn)), x[:, hq + hk:].astype(np.float32)]
    at = host(slots)
    live = (np.arange(n) < used) & (at >= 0)
    for pool, row, factor in zip(pools, rows, (0.5, 1.0)):
        codes, scales = fp4_oracle.encode(row[live], factor)
        full = [np.zeros((blocks * bs, hk, d), dtype=np.uint8), np.zeros((blocks * bs, hk, d // 16), dtype=np.uint8)]
        full[0][at[live]], full[1][at[live]] = codes, scales
        want_pool = fp4_oracle.pack(full[0].reshape(blocks, bs, hk, d), full[1].reshape(blocks, bs, hk, d // 16))
        assert np.array_equal(host(pool), want_pool)


def test_pools_of_more_than_32_bits(cuda_lib):
    """Every operator on the last blocks of pools of 5 GB, decode steps and a chunk through 16 bits."""
    import torch
    sp = cuda_lib
    bs, d, hk, blocks = 128, 128, 4, 140000
    pools = [torch.zeros(blocks, hk, bs // 8, 9 * d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert pools[0].numel() > 1 << 32
    n = 300
    gen = torch.Generator(device="cuda").manual_seed(0)
    qkv = torch.randn(n, 12, d, device="cuda", generator=gen).bfloat16()
    ids = np.array([blocks - 1, 0, blocks - 3], dtype=np.int32)
    at = dev((ids[:, None].astype(np.int64) * bs + np.arange(bs)).reshape(-1)[:n].astype(np.int32))
    sp.append_kv_fp4(qkv[:, 4:8], qkv[:, 8:], at, *pools)
    back = [sp.unpack_fp4(p, slots=at) for p in pools]
    for x, rows in zip(back, (qkv[:, 4:8], qkv[:, 8:])):
        assert np.array_equal(host(x), fp4_oracle.decode(*fp4_oracle.encode(host(rows).astype(np.float32))))
    sp.copy_kv(pools, i32(blocks - 3, blocks - 1), i32(5, blocks - 7), rows=bs)
    sp.copy_kv(pools, i32(blocks * bs - 1), i32((blocks - 20) * bs + 9))
    assert torch.equal(sp.unpack_fp4(pools[0], slots=i32(blocks * bs - 1)), sp.unpack_fp4(pools[0], slots=i32((blocks - 20) * bs + 9)))
    q, table = qkv[:, :4].contiguous(), dev(np.array([ids, [blocks - 7, 0, 5]], dtype=np.int32))
    pad = [np.concatenate([host(x), np.zeros((3 * bs - n, hk, d))]).reshape(3, bs, hk, d) for x in back]
    for new in (1, 150):
        off = i32(0, new, 2 * new)
        out = sp.paged_attention_fp4(q[:2 * new], off, i32(n, n), table, *pools, max_new=new)
        ref = paged_oracle.paged_attention(host(q[:2 * new]), host(off), [n, n], np.tile(np.arange(3), (2, 1)), *pad)
        check_attention(out, None, ref, [n, n], d, "bf16", 2 * new, 30.0)


def test_a_workspace_serves_smaller_calls(cuda_lib):
    """The largest of several, used for all of them in turn."""
    import torch
    from tests.fp4_cases import fp4_case
    sp = cuda_lib
    cases = [fp4_case(20 + i, ctx, new, 8, 2, d, 16, "fp16") for i, (ctx, new, d) in enumerate(
        [([700, 30], [400, 1], 128), ([2000], [1], 128), ([100, 9], [90, 3], 64), ([40], [40], 256)])]
    ws = max((sp.make_attention_fp4_workspace(c["q"], 3, c["k_pool"], kv_tokens=1 << 16) for c in cases), key=lambda w: w.numel())
    args = [(c["q"], c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"]) for c in cases]
    want = [sp.paged_attention_fp4(*a) for a in args]
    for _ in range(3):
        for a, w in zip(args, want):
            ws.buffer[256:].fill_(0xff)   # (what earlier calls left there counts for nothing)
            assert torch.equal(sp.paged_attention_fp4(*a, ws=ws), w)
    assert sp.device_status(ws) == 0


@pytest.mark.parametrize("fp4", [False, True])
def test_copies_within_a_captured_step(cuda_lib, fp4):
    """The count, the entries and the tables are read when the graph runs."""
    import torch
    sp = cuda_lib
    bs, hk, d, blocks = 16, 2, 64, 12
    gen = torch.Generator(device="cuda").manual_seed(4)
    if fp4:
        pools = [torch.randint(0, 256, (blocks, hk, bs // 8, 9 * d // 2), dtype=torch.uint8, device="cuda", generator=gen)]
    else:
        pools = [torch.randn(blocks, bs, hk, d, device="cuda", generator=gen).bfloat16()]
    src, dst, n = i32(0, 0, 0), i32(0, 0, 0), i32(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp.copy_kv(pools, src, dst, n=n)
    look = (lambda p: fp4_oracle.unpack(host(p))) if fp4 else (lambda p: (host(p),))
    want = [x.reshape(blocks * bs, *x.shape[2:]).copy() for x in look(pools[0])]
    for s, t, m in (([3, 40, 5], [100, 17, 8], 2), ([9, -1, 7], [101, 120, -1], 3), ([1, 2, 3], [150, 151, 152], 0),
                    ([50, 51, 52], [180, 181, 182], 99)):
        src.copy_(i32(*s)), dst.copy_(i32(*t)), n.fill_(m)
        graph.replay()
        for i in range(min(m, 3)):
            if s[i] >= 0 and t[i] >= 0:
                for x in want:
                    x[t[i]] = x[s[i]]
        assert all(np.array_equal(x.reshape(y.shape), y, equal_nan=True) for x, y in zip(want, look(pools[0])))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("narrow", [False, True])
def test_short_prompts_by_either_way(cuda_lib, d, narrow):
    """Prompts and chunks of little work: by the table's width from the 4-bit rows or through 16 bits."""
    import torch
    from tests.fp4_cases import fp4_case
    sp = cuda_lib
    c = fp4_case(31, [0, 60, 3], [300, 150, 1], 8, 2, d, 16, "bf16")
    table = c["table"][:, :24].contiguous() if narrow else c["table"]
    lse = torch.full((451, 8), 7.0, device="cuda")
    ws = sp.make_attention_fp4_workspace(c["q"], 3, c["k_pool"])
    out = sp.paged_attention_fp4(c["q"], c["q_off"], c["kv_len"], table, c["k_pool"], c["v_pool"], window=100, lse=lse, ws=ws)
    ref = paged_oracle.paged_attention(host(c["q"]), host(c["q_off"]), host(c["kv_len"]), host(table), np.nan_to_num(c["k"]),
                                       np.nan_to_num(c["v"]), window=100)
    check_attention(out, lse, ref, host(c["kv_len"]), d, "bf16", 451, 30.0)
    assert sp.device_status(ws) == 0


@pytest.mark.parametrize("batch", [64, 65, 130])
@pytest.mark.parametrize("room", [None, 900])
def test_chunks_among_many_requests(cuda_lib, batch, room):
    """Layouts of the 16-bit copies by a warp and by a block, with and without room for all of them."""
    import torch
    from tests.fp4_cases import fp4_case
    sp = cuda_lib
    rng = np.random.default_rng(batch)
    new = [int(x) for x in rng.choice([0, 1, 1, 2, 70], batch)]
    for i in (0, 33, batch - 1):
        new[i] = 100 + i
    ctx = [int(x) for x in rng.integers(0, 300, batch)]
    c = fp4_case(batch, ctx, new, 4, 1, 64, 32, "fp16")
    ws = sp.make_attention_fp4_workspace(c["q"], batch, c["k_pool"], kv_tokens=room)
    for _ in range(2):
        out = sp.paged_attention_fp4(c["q"], c["q_off"], c["kv_len"], c["table"], c["k_pool"], c["v_pool"], ws=ws)
    ref = paged_oracle.paged_attention(host(c["q"]), host(c["q_off"]), host(c["kv_len"]), host(c["table"]), np.nan_to_num(c["k"]),
                                       np.nan_to_num(c["v"]))
    check_attention(out, None, ref, host(c["kv_len"]), 64, "fp16", sum(new), 30.0)
    assert sp.device_status(ws) == 0


@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 16, 4), (256, 6, 2)])
@pytest.mark.parametrize("batch,top", [(1, 380), (9, 200), (70, 380), (300, 64)])
def test_rows_that_hold_short_contexts(cuda_lib, d, hq, hk, batch, top):
    """By a table that holds no context long enough to be cut the results are those of a wide one, bit for bit."""
    import torch
    from tests.fp4_cases import fp4_case
    sp = cuda_lib
    rng = np.random.default_rng(batch)
    new = [int(x) for x in rng.choice([0, 1, 1, 3], batch)]
    new[0] = 1
    c = fp4_case(batch + d, [int(x) for x in rng.integers(0, top - 3, batch)], new, hq, hk, d, 16, "bf16")
    narrow = c["table"][:, :-(-top // 16)].contiguous()
    got = []
    for table in (narrow, c["table"]):
        lse = torch.full((sum(new), hq), 7.0, device="cuda")
        ws = sp.make_attention_fp4_workspace(c["q"], batch, c["k_pool"], max_new=3)
        out = sp.paged_attention_fp4(c["q"], c["q_off"], c["kv_len"], table, c["k_pool"], c["v_pool"], lse=lse, max_new=3, ws=ws)
        assert sp.device_status(ws) == 0
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    ref = paged_oracle.paged_attention(host(c["q"]), host(c["q_off"]), host(c["kv_len"]), host(narrow), np.nan_to_num(c["k"]),
                                       np.nan_to_num(c["v"]))
    check_attention(*got[0], ref, host(c["kv_len"]), d, "bf16", sum(new), 30.0)
