"""GPU parity of paged_attention where every group of 16 keys carries weight:
many key tiles for each CTA, last tiles that end inside, parts joined from many
CTAs, windows whose edges lie on such keys, a scale of the caller's."""

import pytest

from oracle import paged_oracle
from tests.paged_signals import TILE, check_signals, signal_arrays

pytestmark = pytest.mark.gpu


def _check(sp, ctx, new, hq, hk, d, bs, dtype, seed, scale=0.0, **kw):
    import torch

    from tests.paged_cases import torch_dtype
    a = signal_arrays(seed, ctx, new, hq, hk, d, bs, dtype)
    if scale:   # the same logits by another way
        a["q"] = a["q"] * 0.5
        kw["scale"] = scale
    t = {n: torch.from_numpy(x).cuda() for n, x in a.items()}
    q, k_pool, v_pool = [t[n].to(torch_dtype(dtype)) for n in ("q", "k_pool", "v_pool")]
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float32, device="cuda")
    ws = sp.make_attention_workspace(q, len(ctx), k_pool)
    sp.paged_attention(q, t["q_off"], t["kv_len"], t["table"], k_pool, v_pool, out=out, lse=lse, ws=ws, **kw)
    assert sp.device_status(ws) == 0
    ref = paged_oracle.paged_attention(a["q"], a["q_off"], a["kv_len"], a["table"], a["k_pool"], a["v_pool"], **kw)
    check_signals(out, lse, ref, a["kv_len"], d, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,hq,hk", [(64, 6, 2), (128, 4, 1), (256, 8, 2)])
def test_a_few_tokens_over_a_long_context(cuda_lib, d, hq, hk, dtype):
    _check(cuda_lib, [32768], [8], hq, hk, d, 16, dtype, d)
    _check(cuda_lib, [16383], [1], hq, hk, d, 64, dtype, d + 1)


@pytest.mark.parametrize("d,hq,hk", [(64, 6, 2), (128, 16, 4), (256, 8, 2)])
def test_single_tokens_over_long_contexts(cuda_lib, d, hq, hk):
    _check(cuda_lib, [6001, 12000, 16383, 4097, 8200, 777, 127, 128], [1, 1, 1, 1, 3, 1, 1, 1], hq, hk, d, 16, "bf16", d)


@pytest.mark.parametrize("d,hq,hk", [(64, 3, 1), (128, 4, 1), (256, 2, 1)])
def test_chunks_over_long_contexts(cuda_lib, d, hq, hk):
    _check(cuda_lib, [9000, 0, 2500], [200, 700, 1], hq, hk, d, 128, "bf16", d)
    _check(cuda_lib, [4000], [333], hq, hk, d, 8, "fp16", d, causal=False)


@pytest.mark.parametrize("d,hq,hk", [(64, 6, 2), (128, 4, 1), (256, 4, 2)])
def test_windows_whose_edge_is_a_signal(cuda_lib, d, hq, hk):
    for window in (20000 + 1 - 100 * TILE, 20000 + 1 - 99 * TILE + 1, TILE, 20000):
        _check(cuda_lib, [20000], [9], hq, hk, d, 32, "bf16", window, window=window)


def test_a_batch_laid_out_by_its_own_kernel(cuda_lib):
    """More requests than a CTA lays out by itself, some of them long."""
    ctx = [7 * (i % 90) for i in range(500)]
    ctx[3] = ctx[250] = ctx[499] = 9001
    _check(cuda_lib, ctx, [1 + (i % 7 == 0) for i in range(500)], 4, 2, 64, 16, "bf16", 5)


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "bf16")])
def test_a_scale_of_the_callers(cuda_lib, d, dtype):
    _check(cuda_lib, [5000, 3], [4, 150], 4, 2, d, 16, dtype, d, scale=2.0 * d ** -0.5)
    _check(cuda_lib, [700], [60], 4, 2, d, 16, dtype, d, scale=0.01)
