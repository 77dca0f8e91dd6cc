"""GPU tests of paged_attention's slow path (rows masked from a value that is
infinite or NaN are taken again one by one) where it lasts longer than a device
wait may: the other warps' waits do not run out meanwhile."""

import numpy as np
import pytest

from oracle import paged_oracle
from tests.paged_cases import check_attention, host, torch_dtype

pytestmark = pytest.mark.gpu

# Polls of a wait: some 20 ms, where a call without the slow path takes less than
# one and the slow path's rows over 40,000 keys some hundreds.
SPIN = 1 << 14


@pytest.mark.parametrize("d,dtype,value", [(64, "bf16", float("nan")), (128, "fp16", float("inf")),
                                           (256, "bf16", float("nan"))])
def test_rows_taken_again_outlast_the_waits(cuda_lib, d, dtype, value):
    """160 requests of three new tokens over the same 40,000 cached ones, more
    than there are SMs: most CTAs end one request and begin another. In three
    of them the second new token's value has a column that is no number."""
    import torch
    sp = cuda_lib
    n, new, ctx, bs, hq = 160, 3, 40000, 64, 4
    shared = ctx // bs
    rng = np.random.default_rng(d)
    dt = torch_dtype(dtype)
    pools = [torch.from_numpy(rng.standard_normal((shared + n, bs, 1, d), dtype=np.float32)).cuda().to(dt)
             for _ in range(2)]
    table = np.concatenate([np.tile(rng.permutation(shared), (n, 1)), shared + np.arange(n)[:, None]], 1)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    q = torch.from_numpy(rng.standard_normal((n * new, hq, d), dtype=np.float32)).cuda().to(dt)
    off, kv, tab = i32(np.arange(n + 1) * new), i32(np.full(n, ctx + new)), i32(table)
    ws = sp.make_attention_workspace(q, n, pools[0])

    def call(spin):
        out, lse = torch.zeros_like(q), torch.zeros(n * new, hq, device="cuda")
        sp.paged_attention(q, off, kv, tab, *pools, out=out, lse=lse, ws=ws, spin_limit=spin)
        return sp.device_status(ws), out, lse

    status, clean, clean_lse = call(SPIN)
    assert status == 0
    bad, col = [3, 80, 159], d - 3
    pools[1][[shared + b for b in bad], 1, 0, col] = value
    status, out, lse = call(SPIN)
    assert status == 0
    # requests without such a value: the same bits
    good = torch.ones(n * new, dtype=torch.bool, device="cuda")
    for b in bad:
        good[b * new:(b + 1) * new] = False
    assert torch.equal(out[good], clean[good]) and torch.equal(lse[good], clean_lse[good])
    # the others: the tokens that see the value have no number in its column, all else is as without it
    rows = np.concatenate([np.arange(b * new, (b + 1) * new) for b in bad])
    o = host(out)[rows].reshape(len(bad), new, hq, d)
    assert not np.isfinite(o[:, 1:, :, col]).any() and np.isfinite(o[:, 0]).all()
    pools[1][[shared + b for b in bad], 1, 0, col] = 0
    ref = paged_oracle.paged_attention(host(q)[rows], np.arange(len(bad) + 1) * new, [ctx + new] * len(bad), table[bad],
                                       *[host(p) for p in pools])
    fixed = out[torch.from_numpy(rows).cuda()].clone().reshape(len(bad), new, hq, d)
    fixed[:, 1:, :, col] = torch.from_numpy(ref[0]).reshape(o.shape)[:, 1:, :, col].to(dt).cuda()
    check_attention(fixed.reshape(-1, hq, d), lse[torch.from_numpy(rows).cuda()], ref, [ctx + new], d, dtype, len(rows))
