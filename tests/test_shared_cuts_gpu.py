"""Requests cut inside blocks that others hold as well."""

import numpy as np
import pytest

from oracle import fp4_oracle
from tests.fp4_cases import dev
from tests.paged_cases import host
from tests.test_pages_gpu import fork, i32, pages_case

pytestmark = pytest.mark.gpu


def free(c, new, status, alone):
    import speculative_prefill_token_gb300 as sp
    sh, fr = dev(c["shared"]), dev(c["free"])
    out = sp.free_blocks(i32(c["ctx"]), i32(new), dev(c["table"]), sh, fr, i32(c["n_free"]), c["bs"], status=status, alone=alone)
    return [host(x) for x in out], host(sh), host(fr)


@pytest.mark.parametrize("parents,forks,lo,hi,bs", [(1, 1, 40, 40, 16), (40, 3, 0, 300, 8), (1500, 2, 0, 40, 8), (6, 2, 1, 90, 3)])
def test_cuts_inside_shared_blocks_are_refused_on_request(parents, forks, lo, hi, bs):
    import torch
    rng = np.random.default_rng(parents + bs)
    c = pages_case(parents + forks, parents, forks, lo, hi, bs)
    (kv, _, _, left), table, shared = fork(c)
    c.update(ctx=kv, table=table, shared=shared, n_free=int(left[0]))
    some = rng.random(len(kv)) < 0.3
    ends = np.where(some, 0, kv)                                         # requests that end
    fits = np.where(some, kv - kv % bs, kv)                              # cuts between blocks
    own = np.where(some & (kv % bs > 1), kv - kv % bs + 1, kv)           # within the begun block, of one holder
    families = dict(zip(c["dst"].tolist(), c["src"].tolist()))
    root = np.array([families.get(b, b) for b in range(len(kv))])
    whole = np.isin(root, root[some])
    last = np.where(whole, 0, kv)                                        # all holders of a block but one end, which is cut
    last[root[some]] = np.maximum(kv[root[some]] - bs - 1, 0)
    for new in (ends, fits, own, last):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        want = fp4_oracle.free_blocks(c["ctx"], new, c["table"], c["shared"], c["free"], c["n_free"], bs)
        (got_kv, got_left), got_shared, got_free = free(c, new, status, alone=True)
        assert int(status) == 0
        assert np.array_equal(got_kv, want[0]) and got_left[0] == want[1]
        assert np.array_equal(got_shared, want[2]) and np.array_equal(got_free, want[3])
    # one request alone is cut inside a full block that its family shares
    b = int(np.flatnonzero((kv >= bs) & (kv == kv.max()))[0])
    new = np.where(some & (np.arange(len(kv)) != b) & (root != root[b]), 0, kv)
    new[b] = kv[b] // bs * bs - bs + 1
    assert shared[table[b, new[b] // bs]] > 0
    for alone, code in ((True, 6), (False, 0)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        (got_kv, got_left), got_shared, got_free = free(c, new, status, alone=alone)
        assert int(status) == code
        if alone:
            assert np.array_equal(got_kv, kv) and got_left[0] == c["n_free"]
            assert np.array_equal(got_shared, c["shared"]) and np.array_equal(got_free, c["free"])
        else:
            assert np.array_equal(got_kv, new)


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
def test_a_request_cut_inside_a_shared_block_goes_on_in_a_row_of_its_own(dtype):
    """Cut, forked into an empty row, the cut row freed, filled further: the other holder's rows stay."""
    import torch

    import speculative_prefill_token_gb300 as sp
    bs, hk, d, blocks, n = 16, 2, 64, 12, 44
    gen = torch.Generator(device="cuda").manual_seed(3)
    if dtype == "fp4":
        pools = [sp.make_pool_fp4(blocks, bs, hk, d) for _ in range(2)]
        append, rows = sp.append_kv_fp4, lambda s: [sp.unpack_fp4(p, slots=s) for p in pools]
    else:
        pools = [torch.zeros(blocks, bs, hk, d, device="cuda").bfloat16() for _ in range(2)]
        append, rows = sp.append_kv, lambda s: [p.view(-1, hk, d)[s.long()] for p in pools]
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    list_, shared, status = i32(np.arange(blocks)), i32(np.zeros(blocks)), i32(0)

    def fill(ctx, off, left, kv):
        slots, ctx, left = sp.block_tables(ctx, off, list_, left, table, bs, n_tokens=kv.shape[0], status=status)
        append(kv[:, :hk], kv[:, hk:], slots, *pools, status=status)
        return ctx, left

    def cached(b, length):
        at = host(table)[b, np.arange(length) // bs] * bs + np.arange(length) % bs
        return rows(i32(at))

    kv = lambda m: torch.randn(m, 2 * hk, d, device="cuda", generator=gen).bfloat16()  # noqa: E731
    ctx, left = fill(i32([0, 0, 0]), i32([0, n, n, n]), i32(blocks), kv(n))
    ctx, cs, cd, left = sp.fork_blocks(i32(0), i32(1), ctx, table, shared, list_, left, bs, status=status)
    sp.copy_kv(pools, cs, cd, rows=bs, status=status)
    before = cached(0, n)
    # request 1 is cut to 20 tokens, inside the second block, which request 0 holds too
    assert host(sp.free_blocks(ctx, i32([n, 20, 0]), table, shared.clone(), list_.clone(), left, bs, status=i32(0), alone=True)[0]).tolist() == [n, n, 0]
    ctx, left = sp.free_blocks(ctx, i32([n, 20, 0]), table, shared, list_, left, bs, status=status)
    ctx, cs, cd, left = sp.fork_blocks(i32(1), i32(2), ctx, table, shared, list_, left, bs, status=status)
    sp.copy_kv(pools, cs, cd, rows=bs, status=status)
    ctx, left = sp.free_blocks(ctx, i32([n, 0, 20]), table, shared, list_, left, bs, status=status)
    ctx, left = fill(ctx, i32([0, 0, 0, 21]), left, kv(21))
    assert int(status) == 0 and host(ctx).tolist() == [n, 0, 41]
    after, other = cached(0, n), cached(2, 41)
    for x, y, z in zip(before, after, other):
        assert torch.equal(x, y) and torch.equal(x[:20], z[:20]) and not torch.equal(x[20:41], z[20:])
    ctx, left = sp.free_blocks(ctx, i32([0, 0, 0]), table, shared, list_, left, bs, status=status)
    assert int(status) == 0 and int(left) == blocks and not shared.any()
