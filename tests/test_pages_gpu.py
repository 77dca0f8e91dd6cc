"""Forks, frees and copies of cache pages against plain loops."""

import numpy as np
import pytest

from oracle import fp4_oracle
from tests.fp4_cases import dev
from tests.paged_cases import host

pytestmark = pytest.mark.gpu


def i32(v):
    return dev(np.asarray(v, dtype=np.int32).reshape(-1))


def pages_case(seed, parents, forks, lo, hi, bs, idle=0.0, spare=None, width=None):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(lo, hi + 1, parents)
    held = -(-ctx // bs)
    spare = parents * forks + 3 if spare is None else spare
    pool = int(held.sum()) + spare
    ids = rng.permutation(pool)
    rows = parents * (forks + 1)
    width = max(int(held.max(initial=1)), 1) + 2 if width is None else width
    table = np.full((rows, width), -9, dtype=np.int32)
    order = rng.permutation(rows)
    first = 0
    for r, n in zip(order, held):
        table[r, :n] = ids[first:first + n]
        first += n
    ctx_len = np.zeros(rows, dtype=np.int32)
    ctx_len[order[:parents]] = ctx
    src = np.repeat(order[:parents], forks)
    src = np.where(rng.random(src.size) < idle, -1, src)
    free = np.full(pool + 4, -5, dtype=np.int32)
    free[:spare] = ids[first:]
    return dict(src=src, dst=order[parents:], ctx=ctx_len, table=table, shared=np.zeros(pool, dtype=np.int32), free=free,
                n_free=spare, bs=bs)


def fork(c, status=None):
    import speculative_prefill_token_gb300 as sp
    t, sh = dev(c["table"]), dev(c["shared"])
    out = sp.fork_blocks(i32(c["src"]), i32(c["dst"]), i32(c["ctx"]), t, sh, i32(c["free"]), i32(c["n_free"]), c["bs"],
                         status=status)
    return [host(x) for x in out], host(t), host(sh)


@pytest.mark.parametrize("parents,forks,lo,hi,bs", [(1, 1, 5, 5, 8), (1, 4, 4000, 4000, 16), (3, 1, 0, 0, 16), (40, 7, 0, 700, 32),
                                                    (1, 3, 64, 64, 64), (2, 900, 1, 300, 128), (1500, 2, 0, 40, 8), (5, 3, 1, 900, 3)])
def test_forks(parents, forks, lo, hi, bs):
    import torch
    c = pages_case(parents + forks, parents, forks, lo, hi, bs, idle=0.1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    (kv, cs, cd, left), table, shared = fork(c, status)
    want = fp4_oracle.fork_blocks(c["src"], c["dst"], c["ctx"], c["table"], c["shared"], c["free"], c["n_free"], bs)
    assert int(status) == 0
    for got, ref in zip((kv, cs, cd, left[0], table, shared), want):
        assert np.array_equal(got, ref)


def broken(c, **change):
    return dict(c, **{k: np.array(v) for k, v in change.items() if not isinstance(v, int)},
                **{k: v for k, v in change.items() if isinstance(v, int)})


def test_forks_that_are_refused_on_the_device():
    import torch
    base = pages_case(7, 3, 2, 20, 60, 16)
    src, dst, ctx = base["src"], base["dst"], base["ctx"]
    cases = [(7, broken(base, n_free=int((ctx[src] % 16 != 0).sum()) - 1))]
    cases += [(6, broken(base, n_free=-1)), (6, broken(base, n_free=len(base["free"]) + 1))]
    cases += [(6, broken(base, src=np.r_[src[:-1], len(ctx)])), (6, broken(base, dst=np.r_[dst[:-1], -1])),
              (6, broken(base, dst=np.r_[dst[:-1], len(ctx)])), (6, broken(base, dst=np.r_[dst[:-1], dst[0]])),
              (6, broken(base, dst=np.r_[dst[:-1], src[0]])), (6, broken(base, src=np.r_[src[:-1], dst[0]]))]
    long = ctx.copy()
    long[src[0]] = 100000
    neg = ctx.copy()
    neg[src[0]] = -1
    held = ctx.copy()
    held[dst[0]] = 1
    cases += [(6, broken(base, ctx=x)) for x in (long, neg, held)]
    for code, c in cases:
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        (kv, cs, cd, left), table, shared = fork(c, status)
        assert int(status) == code
        assert np.array_equal(table, c["table"]) and np.array_equal(shared, c["shared"]) and np.array_equal(kv, c["ctx"])
        assert (cs == -1).all() and (cd == -1).all() and left[0] == c["n_free"]


def free(c, new, status=None, **more):
    import speculative_prefill_token_gb300 as sp
    sh, fr = dev(c["shared"]), dev(c["free"])
    out = sp.free_blocks(i32(c["ctx"]), i32(new), dev(c["table"]), sh, fr, i32(c["n_free"]), c["bs"], status=status)
    return [host(x) for x in out], host(sh), host(fr)


@pytest.mark.parametrize("parents,forks,lo,hi,bs", [(1, 1, 5, 5, 8), (1, 4, 4000, 4000, 16), (40, 7, 0, 700, 32), (2, 200, 1, 300, 128),
                                                    (1500, 2, 0, 40, 8), (300, 3, 0, 3000, 8), (4, 2, 1, 900, 3)])
def test_frees_after_forks(parents, forks, lo, hi, bs):
    import torch
    rng = np.random.default_rng(parents)
    c = pages_case(parents + forks, parents, forks, lo, hi, bs)
    (kv, _, _, left), table, shared = fork(c)
    c.update(ctx=kv, table=table, shared=shared, n_free=int(left[0]))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # some end, some are cut, some stay; then all the others end
    u = rng.random(len(kv))
    new = np.where(u < 0.4, 0, np.where(u < 0.7, (kv * rng.random(len(kv))).astype(int), kv))
    for target in (new, np.zeros_like(kv)):
        want = fp4_oracle.free_blocks(c["ctx"], target, c["table"], c["shared"], c["free"], c["n_free"], bs)
        (kv, left), shared, fr = free(c, target, status)
        assert int(status) == 0
        assert np.array_equal(kv, want[0]) and left[0] == want[1]
        assert np.array_equal(shared, want[2]) and np.array_equal(fr, want[3])
        c.update(ctx=kv, shared=shared, free=fr, n_free=int(left[0]))
    assert c["n_free"] == len(c["shared"]) and not c["shared"].any()
    assert sorted(c["free"][:c["n_free"]]) == list(range(len(c["shared"])))


def test_large_pool():
    """Several steps of every slice, the last one short."""
    rng = np.random.default_rng(0)
    pool, rows, width = 150_001, 300, 400
    table = rng.permutation(pool)[:rows * width].reshape(rows, width).astype(np.int32)
    c = dict(ctx=np.full(rows, width * 8), table=table, shared=np.zeros(pool, dtype=np.int32),
             free=np.full(pool, -1, dtype=np.int32), n_free=7, bs=8)
    new = rng.integers(0, width * 8 + 1, rows)
    want = fp4_oracle.free_blocks(c["ctx"], new, table, c["shared"], c["free"], 7, 8)
    (kv, left), shared, fr = free(c, new)
    assert left[0] == want[1] and np.array_equal(fr, want[3]) and np.array_equal(shared, want[2])


def test_frees_that_are_refused_on_the_device():
    import torch
    c = pages_case(9, 4, 0, 100, 300, 16, spare=5)
    zero = np.zeros_like(c["ctx"])
    longer = c["ctx"] + 1
    twice = dict(c, table=c["table"].copy())
    twice["table"][1, 0] = twice["table"][0, 0]     # held once, let go twice
    short = dict(c, free=c["free"][:8])
    for code, case, new in ((6, c, longer), (6, c, zero - 1), (6, dict(c, n_free=-1), zero), (6, dict(c, n_free=10000), zero),
                            (6, dict(c, ctx=c["ctx"] + 100000), c["ctx"]), (6, twice, zero), (7, short, zero)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        (kv, left), shared, fr = free(case, new, status)
        assert int(status) == code
        assert np.array_equal(kv, case["ctx"]) and left[0] == case["n_free"]
        assert np.array_equal(shared, case["shared"]) and np.array_equal(fr, case["free"])


def test_bad_block_ids_are_counted_nowhere():
    import torch
    c = pages_case(10, 2, 1, 40, 60, 8)
    c["table"][c["src"][0], 1] = 1 << 20
    c["table"][c["src"][1], 2] = -3
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    (kv, _, _, left), table, shared = fork(c, status)
    assert int(status) == 6 and shared.sum() == (c["ctx"][c["src"]] // 8).sum() - 2
    status.zero_()
    c.update(ctx=kv, table=table, shared=shared, n_free=int(left[0]))
    (kv, left), shared, fr = free(c, np.zeros_like(kv), status)
    assert int(status) == 6 and not kv.any()
    assert left[0] == len(shared) - 2 and not shared.any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp4"])
@pytest.mark.parametrize("d,hk,bs", [(64, 1, 8), (128, 3, 16), (256, 2, 128)])
@pytest.mark.parametrize("n_pools", [1, 5])
def test_copies(dtype, d, hk, bs, n_pools):
    import torch

    import speculative_prefill_token_gb300 as sp
    rng = np.random.default_rng(d + bs)
    blocks = 30
    shape = (blocks, hk, bs // 8, 9 * d // 2) if dtype == "fp4" else (blocks, bs, hk, d)
    pools = []
    for _ in range(n_pools):
        x = torch.randint(-2 ** 15, 2 ** 15, shape, device="cuda", dtype=torch.int16)
        pools.append(x.to(torch.uint8) if dtype == "fp4" else x.view({"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]))
    bits = lambda p: p.cpu().numpy() if dtype == "fp4" else p.view(torch.int16).cpu().numpy()  # noqa: E731

    def rows_of(a):   # [slots, ...] views of everything a slot holds
        if dtype != "fp4":
            return [a.reshape(blocks * bs, hk, d)]
        return [x.reshape(blocks * bs, *x.shape[2:]) for x in fp4_oracle.unpack(a)]

    def back(rows):
        if dtype != "fp4":
            return rows[0].reshape(shape)
        return fp4_oracle.pack(*[x.reshape(blocks, bs, *x.shape[1:]) for x in rows])

    # whole blocks, some entries idle
    perm = rng.permutation(blocks)
    src, dst = perm[:12].copy(), perm[12:24].copy()
    src[3] = dst[5] = -1
    before = [bits(p) for p in pools]
    sp.copy_kv(pools, i32(src), i32(dst), rows=bs)
    for p, old in zip(pools, before):
        want = old.copy()
        m = (src >= 0) & (dst >= 0)
        want[dst[m]] = old[src[m]]
        assert np.array_equal(bits(p), want)
    # single tokens
    slots = rng.permutation(blocks * bs)
    n = blocks * bs // 3
    src, dst = slots[:n].copy(), slots[n:2 * n].copy()
    dst[1] = -1
    before = [bits(p) for p in pools]
    sp.copy_kv(pools, i32(src), i32(dst), n=i32([n - 2]))
    for p, old in zip(pools, before):
        rows = [x.copy() for x in rows_of(old)]
        m = (dst >= 0) & (np.arange(n) < n - 2)
        for x, y in zip(rows, rows_of(old)):
            x[dst[m]] = y[src[m]]
        assert np.array_equal(bits(p), back(rows))


@pytest.mark.parametrize("batch", [1, 3, 40, 1200])
def test_kept_tokens_move_to_blocks_of_their_own(batch):
    """Requests of a table, empty ones among them; entries behind the last offset are not used."""
    import torch

    import speculative_prefill_token_gb300 as sp
    rng = np.random.default_rng(batch)
    bs, hk, d = 16, 2, 64
    ctx = rng.integers(0, 70, batch)
    ctx[0] = 70
    held = -(-ctx // bs)
    width = 6
    blocks = int(held.sum())
    table = np.full((batch, width), -1, dtype=np.int32)
    ids, first = rng.permutation(blocks), 0
    for b, n in enumerate(held):
        table[b, :n] = ids[first:first + n]
        first += n
    keep = [np.sort(rng.permutation(int(c))[:rng.integers(0, int(c) + 1)]) for c in ctx]
    off = np.concatenate([[0], np.cumsum([len(k) for k in keep])])
    flat = np.concatenate(keep + [np.zeros(5, dtype=int)])
    n = int(off[-1])
    total = blocks + -(-n // bs) + 1
    pools = [torch.randn(total, bs, hk, d, device="cuda").bfloat16() for _ in range(2)]
    dst = np.concatenate([blocks * bs + rng.permutation(n), np.zeros(5, dtype=int)])
    before = [p.clone() for p in pools]
    sp.copy_kv(pools, i32(flat), i32(dst), block_table=dev(table), src_off=i32(off))
    for p, old in zip(pools, before):
        want = old.view(-1, hk, d).clone()
        for b, k in enumerate(keep):
            at = table[b, k // bs] * bs + k % bs
            want[torch.from_numpy(dst[off[b]:off[b + 1]]).cuda()] = old.view(-1, hk, d)[torch.from_numpy(at).long().cuda()]
        assert torch.equal(p.view(-1, hk, d), want)


def test_copies_out_of_range_are_skipped():
    import torch

    import speculative_prefill_token_gb300 as sp
    pool = torch.randn(4, 8, 1, 64, device="cuda").bfloat16()
    old = pool.clone()
    for src, dst, more in (([32], [0], {}), ([0], [32], {}), ([4], [0], dict(rows=8)), ([0], [4], dict(rows=8)),
                           ([8], [0], dict(block_table=dev(np.array([[1]], dtype=np.int32)), src_off=i32([0, 1]))),
                           ([0], [0], dict(block_table=dev(np.array([[-1]], dtype=np.int32)), src_off=i32([0, 1]))),
                           ([0], [0], dict(block_table=dev(np.array([[4]], dtype=np.int32)), src_off=i32([0, 1])))):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        sp.copy_kv([pool], i32(src), i32(dst), status=status, **more)
        assert int(status) == 6 and torch.equal(pool, old)


def test_strided_pools():
    """Pools of two layers interleaved, heads outside tokens."""
    import torch

    import speculative_prefill_token_gb300 as sp
    big = torch.randn(6, 2, 3, 8, 64, device="cuda").half()      # [blocks, layer, Hk, bs, d]
    old = big.clone()
    pools = [big[:, i].transpose(1, 2) for i in range(2)]
    sp.copy_kv(pools, i32([1, 2]), i32([4, 5]), rows=8)
    want = old.clone()
    want[4:6] = old[1:3]
    assert torch.equal(big, want)
    sp.copy_kv(pools[1:], i32([3, 17]), i32([0, 47]))
    want[0, 1, :, 0] = old[0, 1, :, 3]
    want[5, 1, :, 7] = old[2, 1, :, 1]
    assert torch.equal(big, want)


@pytest.mark.parametrize("d,bs", [(256, 15_000_064), (64, 119_400_064)])
def test_tokens_of_a_block_of_more_than_31_bits(d, bs):
    """A pool of one block and one head is one run of rows, whose last lie more than 2^31 bytes (and 2^32) behind
    the first."""
    import torch

    import speculative_prefill_token_gb300 as sp
    assert bs % 128 == 0 and (bs - 20) * (9 * d // 16) > 1 << 31
    pool = torch.zeros(1, 1, bs // 8, 9 * d // 2, dtype=torch.uint8, device="cuda")
    pool[0, 0, -2:] = torch.randint(1, 120, pool.shape[3:], dtype=torch.uint8, device="cuda")
    far, near = np.arange(bs - 12, bs, 3), np.array([0, 9, 18, 30])
    want = sp.unpack_fp4(pool, slots=i32(far))
    assert want.any(-1).all()
    sp.copy_kv([pool], i32(far), i32(near))
    assert torch.equal(sp.unpack_fp4(pool, slots=i32(near)), want)
    sp.copy_kv([pool], i32(near), i32(far - 1))
    assert torch.equal(sp.unpack_fp4(pool, slots=i32(far - 1)), want) and torch.equal(sp.unpack_fp4(pool, slots=i32(far)), want)
    assert not pool[0, 0, 4:-2].any()


def test_forks_by_two_threads_at_once():
    """Calls whose shared memory differs, through the C ABI (which leaves the interpreter's lock)."""
    import ctypes
    import threading

    import torch

    import speculative_prefill_token_gb300 as sp
    from speculative_prefill_token_gb300 import pages
    lib, failed = sp.load(), []

    def caller(forks, stream):
        rows, i32z = 8192, lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        src, ctx, table, shared, free, n_free = i32z(forks) - 1, i32z(rows), i32z(rows * 4), i32z(64), i32z(64), i32z(1)
        outs = [i32z(rows), i32z(forks), i32z(forks), i32z(1), i32z(1)]
        torch.cuda.synchronize()
        shape = pages._PagesShape(n_seqs=rows, n_forks=forks, block_size=16, table_stride=4, pool_blocks=64, free_capacity=64)
        ptr = [t.data_ptr() for t in (src, src.clone(), ctx, table, shared, free, n_free, *outs)]
        torch.cuda.synchronize()
        for _ in range(3000):
            rc = lib.sp_fork_blocks(ctypes.byref(shape), *ptr, stream.cuda_stream)
            if rc:
                failed.append((forks, rc))
                break
        stream.synchronize()
        if int(outs[4]):
            failed.append((forks, "status"))

    streams = [torch.cuda.Stream() for _ in range(2)]
    threads = [threading.Thread(target=caller, args=a) for a in zip((16384, 6500), streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_tables_by_two_threads_at_once():
    import ctypes
    import threading

    import torch

    import speculative_prefill_token_gb300 as sp
    from speculative_prefill_token_gb300 import paged
    lib, failed = sp.load(), []

    def caller(rows, stream):
        i32z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        bufs = [i32z(rows), i32z(rows + 1), i32z(16), i32z(1), i32z(rows * 2), i32z(8), i32z(rows), i32z(1), i32z(1)]
        torch.cuda.synchronize()
        shape = paged._BlockShape(n_seqs=rows, block_size=16, table_stride=2, n_tokens=8, free_capacity=16, pool_blocks=16)
        ptr = [t.data_ptr() for t in bufs]
        for _ in range(3000):
            rc = lib.sp_block_tables(ctypes.byref(shape), *ptr, stream.cuda_stream)
            if rc:
                failed.append((rows, rc))
                break
        stream.synchronize()
        if int(bufs[-1]):
            failed.append((rows, "status"))

    streams = [torch.cuda.Stream() for _ in range(2)]
    threads = [threading.Thread(target=caller, args=a) for a in zip((16384, 4200), streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
