"""GPU tests of block_tables and append_kv against the oracle, and of a whole
step of the target: scoring, block tables, rotation and store, attention."""

import numpy as np
import pytest

from oracle import paged_oracle
from tests.paged_cases import HALF_STEP, check_attention, host, torch_dtype

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _tables_case(seed, ctx, new, bs, spare=4, free_pad=3):
    rng = np.random.default_rng(seed)
    held = [-(-c // bs) for c in ctx]
    need = [-(-(c + n) // bs) for c, n in zip(ctx, new)]
    taken = sum(need) - sum(held)
    ids = rng.permutation(sum(need) + spare)
    table = np.full((len(ctx), max(max(need), 1) + 2), -9, dtype=np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    free = ids[at:]
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    assert len(free) == taken + spare
    return off, table, np.concatenate([free, np.full(free_pad, -5)]).astype(np.int32), len(free)


@pytest.mark.parametrize("bs", [1, 8, 16, 24, 64, 256])
@pytest.mark.parametrize("kind", ["decode", "chunks", "first", "many"])
def test_block_tables(cuda_lib, bs, kind):
    sp = cuda_lib
    rng = np.random.default_rng(bs)
    n = {"decode": 33, "chunks": 9, "first": 5, "many": 5000}[kind]
    ctx = np.zeros(n, int) if kind == "first" else rng.integers(0, 600, n)
    new = {"decode": np.ones(n, int), "chunks": rng.integers(0, 400, n), "first": rng.integers(0, 900, n),
           "many": (rng.random(n) < 0.7).astype(int) + (rng.random(n) < 0.05) * 40}[kind]
    off, table, free, n_free = _tables_case(bs, ctx, new, bs)
    cap = int(off[-1]) + 11
    want = paged_oracle.block_tables(ctx, off, free, n_free, table, bs, cap)
    dev = _i32(table)
    status = _i32([0])
    for _ in range(2):   # (the same call again takes the same blocks)
        slots, kv, left = sp.block_tables(_i32(ctx), _i32(off), _i32(free), _i32([n_free]), dev, bs, n_tokens=cap,
                                          status=status, pool_blocks=int(free.size + table.size))
        assert int(status) == 0
        for got, ref in zip((dev, slots, kv, left), want):
            assert np.array_equal(host(got).reshape(np.shape(ref) or (1,)), np.reshape(ref, np.shape(ref) or (1,)))


def test_block_tables_without_new_tokens(cuda_lib):
    sp = cuda_lib
    off, table, free, n_free = _tables_case(1, [5, 0, 16], [0, 0, 0], 8)
    slots, kv, left = sp.block_tables(_i32([5, 0, 16]), _i32(off), _i32(free), _i32([n_free]), _i32(table), 8, n_tokens=3)
    assert host(slots).tolist() == [-1, -1, -1] and host(kv).tolist() == [5, 0, 16] and int(left) == n_free


def test_block_tables_takes_nothing_when_it_cannot_serve_all(cuda_lib):
    """Too few free blocks, a row that is outgrown and inconsistent lengths:
    the status says so, nothing is taken, every slot is -1, kv_len is 0."""
    sp = cuda_lib
    ctx, new, bs = [10, 3, 0], [20, 1, 30], 8
    off, table, free, n_free = _tables_case(2, ctx, new, bs)
    need = int(paged_oracle.block_tables(ctx, off, free, n_free, table, bs, 51)[3])
    exact_fit = n_free - need
    assert paged_oracle.block_tables(ctx, off, free, exact_fit, table, bs, 51)[3] == 0

    def call(ctx=ctx, off=off, n_free=n_free, table=table, cap=51):
        dev, status = _i32(table), _i32([0])
        slots, kv, left = sp.block_tables(_i32(ctx), _i32(off), _i32(free), _i32([n_free]), dev, bs, n_tokens=cap,
                                          status=status)
        return int(status), host(dev), host(slots), host(kv), int(left)

    assert call(n_free=exact_fit)[0] == 0
    for code, kw in ((7, dict(n_free=exact_fit - 1)), (7, dict(n_free=0)), (6, dict(table=table[:, :3])),
                     (6, dict(ctx=[10, -1, 0])), (6, dict(off=[0, 30, 21, 51])), (6, dict(off=[1, 20, 21, 51])),
                     (6, dict(cap=50)), (6, dict(n_free=len(free) + 1)), (6, dict(n_free=-1))):
        status, dev, slots, kv, left = call(**kw)
        assert status == code, kw
        assert np.array_equal(dev, kw.get("table", table)) and (slots == -1).all() and (kv == 0).all(), kw
        assert left == kw.get("n_free", n_free)
    # a bad id in the free list: the tokens of that block get no slot
    bad = free.copy()
    bad[n_free - 1] = 1 << 29
    status = _i32([0])
    slots, _, _ = sp.block_tables(_i32(ctx), _i32(off), _i32(bad), _i32([n_free]), _i32(table), bs, n_tokens=51,
                                  status=status)
    want = paged_oracle.block_tables(ctx, off, bad, n_free, table, bs, 51)[1]
    assert int(status) == 6
    assert np.array_equal(host(slots), np.where(want >= (1 << 29), -1, want))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hk,d,rotary", [(8, 2, 256, 64), (4, 1, 128, 128), (3, 3, 64, 16), (0, 2, 80, 0),
                                            (2, 1, 48, 48), (5, 1, 64, 0)])
@pytest.mark.parametrize("n", [1, 37, 1500])
def test_append_kv(cuda_lib, dtype, hq, hk, d, rotary, n):
    """Rotated queries and keys within the rounding of the type, values and
    unrotated parts bit for bit, other pool rows and slots of -1 untouched."""
    import torch
    sp = cuda_lib
    rng = np.random.default_rng(n + d)
    dt = torch_dtype(dtype)
    fused = torch.from_numpy(rng.standard_normal((n, hq + 2 * hk + 1, d), dtype=np.float32)).cuda().to(dt)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:hq + 2 * hk]
    bs, blocks = 16, -(-n // 16) + 4
    pools = [torch.from_numpy(rng.standard_normal((blocks, bs, hk, d), dtype=np.float32)).cuda().to(dt)
             for _ in range(2)]
    before = [host(p).reshape(-1, hk, d) for p in pools]
    slots = rng.permutation(blocks * bs)[:n].astype(np.int32)
    if n > 1:
        slots[[0, n // 2]] = -1
    used = n - 2 if n > 30 else n
    max_pos = 5000
    pos = np.sort(rng.permutation(max_pos)[:n]).astype(np.int32)
    pos[-1] = max_pos - 1
    cos_sin = None
    if rotary:
        ang = np.arange(max_pos)[:, None] * 1e4 ** (-np.arange(rotary // 2) * 2.0 / rotary)
        cos_sin = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    status = _i32([0])
    q_out = torch.full((n, hq, d), 9.0, dtype=dt, device="cuda") if hq else None
    got = sp.append_kv(k, v, _i32(slots), *pools, q=q if hq else None, q_out=q_out,
                       positions=_i32(pos) if rotary else None,
                       cos_sin=torch.from_numpy(cos_sin).cuda() if rotary else None, n_new=_i32([used]),
                       status=status)
    assert int(status) == 0 and got is q_out
    kr = paged_oracle.rotate(host(k), pos, cos_sin) if rotary else host(k)
    # two products and a sum in fp32, then one rounding (half a subnormal step of fp16 at least)
    u = HALF_STEP[dtype]

    def close(x, ref, size):
        return (np.abs(x - ref) <= u * np.abs(ref) * (1 + 2.0 ** -20) + 3 * 2.0 ** -24 * size + 2.0 ** -25).all()

    def size(x):
        return np.abs(x).max(-1, keepdims=True) * 2

    live = np.arange(n) < used
    st = live & (slots >= 0)
    kp, vp = [host(p).reshape(-1, hk, d) for p in pools]
    assert close(kp[slots[st]], kr[st], size(host(k)[st]))
    assert np.array_equal(vp[slots[st]], host(v)[st])
    if rotary < d:
        assert np.array_equal(kp[slots[st]][..., rotary:], host(k)[st][..., rotary:])
    others = np.ones(blocks * bs, bool)
    others[slots[st]] = False
    assert np.array_equal(kp[others], before[0][others]) and np.array_equal(vp[others], before[1][others])
    if hq:
        qr = paged_oracle.rotate(host(q), pos, cos_sin) if rotary else host(q)
        assert close(host(q_out)[live], qr[live], size(host(q)[live]))
        assert (host(q_out)[~live] == 9.0).all()
        # in place
        want = q_out.clone()
        sp.append_kv(k, v, _i32(slots), *pools, q=q, q_out=q, positions=_i32(pos) if rotary else None,
                     cos_sin=torch.from_numpy(cos_sin).cuda() if rotary else None, n_new=_i32([used]))
        assert torch.equal(q[:used], want[:used])


def test_append_kv_status_of_bad_slots_and_positions(cuda_lib):
    import torch
    sp = cuda_lib
    k = torch.randn(4, 1, 64, device="cuda").bfloat16()
    pools = [torch.zeros(2, 8, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cs = torch.ones(10, 64, device="cuda")
    status = _i32([0])
    sp.append_kv(k, k, _i32([0, 16, 3, -7]), *pools, status=status)
    assert int(status) == 6
    assert torch.equal(pools[0].view(16, 64)[[0, 3]], k[[0, 2], 0]) and pools[0].count_nonzero() == 128
    for pos in ([1, 2, 10, 3], [1, 2, -1, 3]):
        for p in pools:
            p.zero_()
        status.zero_()
        sp.append_kv(k, k, _i32([0, 1, 2, 3]), *pools, positions=_i32(pos), cos_sin=cs, status=status)
        assert int(status) == 6
        rows = pools[1].view(16, 64)
        assert torch.equal(rows[[0, 1, 3]], k[[0, 1, 3], 0]) and (rows[2] == 0).all() and (pools[0].view(16, 64)[2] == 0).all()


@pytest.mark.parametrize("d,rotary,bs", [(128, 128, 16), (256, 64, 64)])
def test_a_step_of_the_target_after_the_selection(cuda_lib, d, rotary, bs):
    """Scoring, block tables from kept_off, rotation to kept_pos and store,
    attention of the kept tokens, then two decode steps, all chained on the
    device; every stage is held to the oracle on its own inputs."""
    import torch

    from tests._cases import random_case
    sp = cuda_lib
    hq, hk, lengths = 8, 2, [900, 0, 37, 1500]
    q, k, off = random_case(77, lengths, 2, hq, hk, d, 4, q_gain=2.0)
    params = sp.SelectionParams(mode="fixed", keep_p=0.3)
    sel = sp.specprefill_score(torch.from_numpy(q.view(np.int16)).cuda(), torch.from_numpy(k.view(np.int16)).cuda(),
                               _i32(off), params)
    ntot, batch = int(off[-1]), len(lengths)
    width, blocks = -(-max(lengths) // bs) + 1, ntot // bs + 20
    rng = np.random.default_rng(1)
    free = _i32(rng.permutation(blocks))
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    pools = [torch.full((blocks, bs, hk, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ang = np.arange(2000)[:, None] * 1e6 ** (-np.arange(rotary // 2) * 2.0 / rotary)
    cos_sin = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    status = _i32([0])
    ctx, n_free = _i32([0] * batch), _i32([blocks])
    gen = torch.Generator(device="cuda").manual_seed(5)
    new_off, positions, n_new, cap = sel.kept_off, sel.kept_pos, sel.n_kept, ntot
    for step in range(3):
        slots, kv, left = sp.block_tables(ctx, new_off, free, n_free, table, bs, n_tokens=cap, status=status,
                                          pool_blocks=blocks)
        qkv = torch.randn(cap, hq + 2 * hk, d, device="cuda", generator=gen).bfloat16()
        qs = sp.append_kv(qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, *pools, q=qkv[:, :hq], positions=positions,
                          cos_sin=cos_sin, n_new=n_new, status=status)
        lse = torch.zeros(cap, hq, device="cuda")
        ws = sp.make_attention_workspace(qs, batch, pools[0])
        out = sp.paged_attention(qs, new_off, kv, table, *pools, lse=lse, ws=ws)
        assert sp.device_status(ws) == 0 and int(status) == 0
        # held to the oracle
        n = int(host(new_off)[-1])
        want = paged_oracle.rotate(host(qkv[:n, :hq]), host(positions)[:n], host(cos_sin))
        assert np.abs(host(qs)[:n] - want).max() <= 2.0 ** -8 * np.abs(want).max() * 1.01
        rows = host(slots)[:n]
        assert (host(slots)[n:] == -1).all() and len(set(rows.tolist())) == n
        kr = paged_oracle.rotate(host(qkv[:n, hq:hq + hk]), host(positions)[:n], host(cos_sin))
        assert np.abs(host(pools[0]).reshape(-1, hk, d)[rows] - kr).max() <= 2.0 ** -8 * np.abs(kr).max() * 1.01
        ref = paged_oracle.paged_attention(host(qs), host(new_off), host(kv), host(table), host(pools[0]),
                                           host(pools[1]))
        check_attention(out, lse, ref, host(kv), d, "bf16", n)
        # the next step: one token for each request, at its prompt's end
        ctx, n_free = kv, left
        new_off = _i32(np.arange(batch + 1))
        positions, n_new, cap = _i32([x + step for x in lengths]), _i32([batch]), batch


def _step_state(lengths, ctx, hq, hk, d, bs, seed):
    """Tensors of a step over a cache that holds ctx[b] tokens of each request,
    for new tokens in a packed buffer of sum(lengths) + 5 rows."""
    import torch
    off, table, free, n_free = _tables_case(seed, ctx, lengths, bs, spare=3)
    rng = np.random.default_rng(seed)
    cap = int(off[-1]) + 5
    blocks = int(max(table.max(), free.max())) + 1
    pools = [torch.from_numpy(rng.standard_normal((blocks, bs, hk, d), dtype=np.float32)).cuda().bfloat16() for _ in range(2)]
    qkv = torch.from_numpy(rng.standard_normal((cap, hq + 2 * hk, d), dtype=np.float32)).cuda().bfloat16()
    pos = np.zeros(cap, np.int32)
    for b, c in enumerate(ctx):
        pos[off[b]:off[b + 1]] = 3 * c + 2 * np.arange(lengths[b])
    ang = np.arange(4000)[:, None] * 1e4 ** (-np.arange(d // 4) * 4.0 / d)
    cs = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    z = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(ctx=_i32(ctx), off=_i32(off), free=_i32(free), n_free=_i32([n_free]), table=_i32(table), pools=pools,
                qkv=qkv, pos=_i32(pos), cs=cs, n_new=_i32([off[-1]]), slots=z(cap), kv=z(len(ctx)), left=z(1),
                status=z(1), q=torch.zeros(cap, hq, d, dtype=torch.bfloat16, device="cuda"),
                out=torch.zeros(cap, hq, d, dtype=torch.bfloat16, device="cuda"), hq=hq, hk=hk, bs=bs, cap=cap)


def _step(sp, s, ws, stream=None):
    hq, hk = s["hq"], s["hk"]
    sp.block_tables(s["ctx"], s["off"], s["free"], s["n_free"], s["table"], s["bs"], slot_map=s["slots"], kv_len=s["kv"],
                    n_left=s["left"], status=s["status"], stream=stream)
    sp.append_kv(s["qkv"][:, hq:hq + hk], s["qkv"][:, hq + hk:], s["slots"], *s["pools"], q=s["qkv"][:, :hq], q_out=s["q"],
                 positions=s["pos"], cos_sin=s["cs"], n_new=s["n_new"], status=s["status"], stream=stream)
    sp.paged_attention(s["q"], s["off"], s["kv"], s["table"], *s["pools"], out=s["out"], ws=ws, stream=stream)


def test_a_captured_step_replayed_with_other_lengths(cuda_lib):
    """The three operators in one graph: replays give the eager call's bits,
    also after the lengths, rows and free blocks were replaced in place."""
    import torch
    sp = cuda_lib
    a = _step_state([40, 1, 0, 300], [100, 513, 7, 0], 8, 2, 128, 16, 1)
    others = [_step_state(n, c, 8, 2, 128, 16, 2 + i) for i, (n, c) in enumerate(
        [([0, 1, 339, 1], [64, 300, 15, 200]), ([341, 0, 0, 0], [90, 0, 600, 1]), ([1, 1, 1, 1], [0, 0, 0, 0])])]
    wide = max(s["table"].shape[1] for s in [a] + others)
    blocks = max(s["pools"][0].shape[0] for s in [a] + others)
    free = max(s["free"].numel() for s in [a] + others)
    for s in [a] + others:   # the capacities of one captured call
        t = torch.full((4, wide), -9, dtype=torch.int32, device="cuda")
        t[:, :s["table"].shape[1]] = s["table"]
        s["table"] = t
        f = torch.full((free,), -5, dtype=torch.int32, device="cuda")
        f[:s["free"].numel()] = s["free"]
        s["free"] = f
        for i, p in enumerate(s["pools"]):
            s["pools"][i] = torch.zeros(blocks, *p.shape[1:], dtype=p.dtype, device="cuda")
            s["pools"][i][:p.shape[0]] = p
        for name in ("qkv", "pos", "slots", "q", "out"):
            x = s[name]
            s[name] = torch.zeros(a["cap"], *x.shape[1:], dtype=x.dtype, device="cuda")
            s[name][:x.shape[0]] = x
    ws = sp.make_attention_workspace(a["q"], 4, a["pools"][0])
    stage = {k: ([p.clone() for p in v] if isinstance(v, list) else v.clone() if torch.is_tensor(v) else v)
             for k, v in a.items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _step(sp, stage, ws)
    for s in [a] + others + [a]:
        fresh = {k: ([p.clone() for p in v] if isinstance(v, list) else v.clone() if torch.is_tensor(v) else v)
                 for k, v in s.items()}
        for k, v in s.items():
            if isinstance(v, list):
                for x, y in zip(stage[k], v):
                    x.copy_(y)
            elif torch.is_tensor(v):
                stage[k].copy_(v)
        g.replay()
        _step(sp, fresh, ws)
        torch.cuda.synchronize()
        assert sp.device_status(ws) == 0 and int(stage["status"]) == 0 and int(fresh["status"]) == 0
        n = int(s["off"][-1])
        for k in ("slots", "kv", "left", "table", "q", "out"):
            assert torch.equal(stage[k], fresh[k]), k
        for x, y in zip(stage["pools"], fresh["pools"]):
            assert torch.equal(x, y)
        assert n == 0 or stage["out"][:n].float().abs().sum() > 0


def test_steps_on_two_streams_at_once(cuda_lib):
    import torch
    sp = cuda_lib
    states = [_step_state([3, 1, 200], [1000, 20, 0], 8, 2, 256, 16, 7), _step_state([1] * 9, [700] * 9, 6, 3, 64, 32, 8)]
    wss = [sp.make_attention_workspace(s["q"], s["ctx"].numel(), s["pools"][0]) for s in states]
    for s, ws in zip(states, wss):
        _step(sp, s, ws)
    torch.cuda.synchronize()
    want = [s["out"].clone() for s in states]
    streams = [torch.cuda.Stream() for _ in states]
    for s in states:
        s["out"].zero_()
    torch.cuda.synchronize()
    for _ in range(5):   # (the same step again takes the same blocks)
        for s, ws, st in zip(states, wss, streams):
            _step(sp, s, ws, stream=st)
    torch.cuda.synchronize()
    for s, ws, w in zip(states, wss, want):
        assert torch.equal(s["out"], w) and sp.device_status(ws) == 0 and int(s["status"]) == 0


@pytest.mark.parametrize("d,rotary", [(1024, 1024), (16, 16), (1024, 16)])
def test_append_kv_smallest_and_largest_rows(cuda_lib, d, rotary):
    import torch
    sp = cuda_lib
    rng = np.random.default_rng(d)
    n, hk = 23, 2
    k, v = [torch.from_numpy(rng.standard_normal((n, hk, d), dtype=np.float32)).cuda().bfloat16() for _ in range(2)]
    pools = [torch.zeros(n, 1, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]   # blocks of one token
    slots, pos = rng.permutation(n).astype(np.int32), rng.integers(0, 100, n).astype(np.int32)
    ang = np.arange(100)[:, None] * 1e4 ** (-np.arange(rotary // 2) * 2.0 / rotary)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    status = _i32([0])
    sp.append_kv(k, v, _i32(slots), *pools, positions=_i32(pos), cos_sin=torch.from_numpy(cs).cuda(), status=status)
    assert int(status) == 0
    got, ref = host(pools[0])[slots, 0], paged_oracle.rotate(host(k), pos, cs)
    # two products and a sum in fp32, one rounding
    size = 2 * np.abs(host(k)).max(-1, keepdims=True)
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -20) + 3 * 2.0 ** -24 * size + 2.0 ** -25).all()
    assert torch.equal(pools[1][_i32(slots).long(), 0], v)
