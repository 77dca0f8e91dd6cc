"""Store into the 4-bit cache and rows read back, bit for bit against the
definition."""

import numpy as np
import pytest

from oracle import fp4_oracle, paged_oracle
from tests.fp4_cases import dev
from tests.paged_cases import HALF_STEP, host, torch_dtype

pytestmark = pytest.mark.gpu


def store_case(seed, n, hq, hk, d, bs, rot, dtype, max_pos=500, gain=1.0):
    import torch
    rng = np.random.default_rng(seed)
    blocks = -(-n // bs) + 2
    perm = rng.permutation(blocks * bs)[:n]
    qkv = dev(rng.standard_normal((n, hq + 2 * hk, d), dtype=np.float32) * gain).to(torch_dtype(dtype))
    pos = rng.integers(0, max_pos, n).astype(np.int32)
    turn = None
    if rot:
        angle = np.arange(max_pos)[:, None] * 1e4 ** (-np.arange(rot // 2) * 2.0 / rot)
        turn = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    old = [rng.integers(0, 256, (blocks, hk, bs // 8, 9 * d // 2), dtype=np.uint8) for _ in range(2)]
    return dict(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], slots=perm.astype(np.int32), pos=pos, turn=turn,
                old=old, pools=[dev(p) for p in old], bs=bs)


def expected(c, factors=(1.0, 1.0), rows=None):
    """The pools' bytes after the store of rows [0, rows) (all)."""
    out = []
    keys = host(c["k"]).astype(np.float32)
    if c["turn"] is not None:
        keys = fp4_oracle.rotate32(keys, c["pos"], c["turn"])
    for old, x, f in zip(c["old"], (keys, host(c["v"]).astype(np.float32)), factors):
        codes, scales = fp4_oracle.unpack(old)
        new = fp4_oracle.encode(x, f)
        m = np.arange(len(c["slots"])) < (len(c["slots"]) if rows is None else rows)
        m &= c["slots"] >= 0
        for part, y in zip((codes, scales), new):
            part[c["slots"][m] // c["bs"], c["slots"][m] % c["bs"]] = y[m]
        out.append(fp4_oracle.pack(codes, scales))
    return out


def store(c, q=True, **more):
    import speculative_prefill_token_gb300 as sp
    turn = c["turn"] is not None
    return sp.append_kv_fp4(c["k"], c["v"], dev(c["slots"]), *c["pools"], q=c["q"] if q else None,
                            positions=dev(c["pos"]) if turn else None, cos_sin=dev(c["turn"]) if turn else None, **more)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 0), (128, 96), (256, 64), (256, 256), (256, 240)])
@pytest.mark.parametrize("n,bs", [(1, 8), (37, 16), (200, 128)])
def test_rows_are_stored_as_defined(dtype, d, rot, n, bs):
    c = store_case(d + rot + n, n, 5, 3, d, bs, rot, dtype)
    q = store(c, k_scale=0.3, v_scale=4.0)
    for got, want in zip(c["pools"], expected(c, (0.3, 4.0))):
        assert np.array_equal(host(got), want)
    ref = host(c["q"])
    if rot:
        ref = paged_oracle.rotate(ref, c["pos"], c["turn"])
    u = HALF_STEP[dtype]
    # rotated in 32 bits (two products and a sum: 2^-22 of the sizes involved), then rounded
    size = np.abs(host(c["q"])).max(-1, keepdims=True) * 2
    assert (np.abs(host(q) - ref) <= 1.01 * u * np.abs(ref) + 2.0 ** -22 * size + 2.0 ** -25).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("gain", [1e-4, 3e-3, 0.05, 30.0, 2000.0, 60000.0])
def test_small_and_large_rows(dtype, gain):
    """Scales at both ends of e4m3: subnormal, least and saturated."""
    if dtype == "fp16" and gain > 3000:
        pytest.skip("outside the type's range")
    c = store_case(3, 64, 1, 2, 128, 64, 64, dtype, gain=gain)
    store(c, q=False)
    for got, want in zip(c["pools"], expected(c)):
        assert np.array_equal(host(got), want)


def test_ties_zeros_infinities_and_nan():
    import torch
    import speculative_prefill_token_gb300 as sp
    x = torch.zeros(6, 1, 64, dtype=torch.bfloat16, device="cuda")
    # the scale is 1 (largest 6): halfway points go to the even code
    ties = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6]
    x[0, 0, :16] = torch.tensor(ties)
    x[1, 0, 16] = float("inf")
    x[2, 0, 32] = float("nan")
    x[3, 0, 48] = float("-inf")
    x[4, 0, 3] = 3.3e38
    x[5, 0] = -0.0
    pool = [sp.make_pool_fp4(1, 8, 1, 64) for _ in range(2)]
    sp.append_kv_fp4(x, x, torch.arange(6, dtype=torch.int32, device="cuda"), *pool)
    codes, scales = fp4_oracle.encode(host(x)[None].astype(np.float32))
    got = fp4_oracle.unpack(host(pool[0]))
    assert np.array_equal(got[0][:, :6], codes) and np.array_equal(got[1][:, :6], scales)
    assert torch.equal(pool[0], pool[1])
    back = sp.unpack_fp4(pool[0])
    assert back[0, 0, 0, :16].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, -6]
    for row, group in ((1, 1), (2, 2), (3, 3)):
        nan = torch.isnan(back[0, row, 0]).view(4, 16)
        assert nan[group].all() and not nan[torch.arange(4) != group].any()
    assert back[0, 4, 0, 3] == 2688.0 and (back[0, 5:] == 0).all()


def test_rows_that_are_not_stored():
    import torch
    c = store_case(5, 40, 2, 2, 64, 16, 64, "bf16")
    c["slots"][3] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    store(c, n_new=dev(np.array([29], dtype=np.int32)), status=status)
    for got, want in zip(c["pools"], expected(c, rows=29)):
        assert np.array_equal(host(got), want)
    assert int(status) == 0
    c = store_case(5, 40, 2, 2, 64, 16, 64, "bf16")
    good = c["slots"].copy()
    c["slots"][7] = c["pools"][0].shape[0] * 16
    c["pos"][9] = 500
    store(c, status=status)
    assert int(status) == 6
    c["slots"][7] = c["slots"][9] = -1
    c["pos"][9] = 0
    for got, want in zip(c["pools"], expected(c)):
        assert np.array_equal(host(got), want)
    assert (good >= 0).all()


def test_in_place_queries_and_strided_pools():
    import torch
    c = store_case(6, 33, 4, 2, 128, 32, 128, "bf16")
    want = store(c)
    wide = [torch.zeros(p.shape[0], 3, *p.shape[1:], dtype=torch.uint8, device="cuda") for p in c["pools"]]
    for w, old in zip(wide, c["old"]):
        w[:, 1] = dev(old)
    d = dict(c, pools=[w[:, 1] for w in wide])
    got = store(d, q_out=c["q"])
    assert got.data_ptr() == c["q"].data_ptr() and torch.equal(got, want)
    for w, p in zip(wide, c["pools"]):
        assert torch.equal(w[:, 1], p) and not w[:, 0].any() and not w[:, 2].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,bs,hk", [(64, 8, 1), (128, 64, 3), (256, 384, 2)])
def test_rows_read_back(dtype, d, bs, hk):
    import torch

    import speculative_prefill_token_gb300 as sp
    rng = np.random.default_rng(d)
    pool = rng.integers(0, 256, (5, hk, bs // 8, 9 * d // 2), dtype=np.uint8)
    codes, scales = fp4_oracle.unpack(pool)
    scales &= 127
    pool = fp4_oracle.pack(codes, scales)
    v = fp4_oracle.values(pool)
    got = sp.unpack_fp4(dev(pool), torch_dtype(dtype))
    assert got.shape == (5, bs, hk, d)
    assert np.array_equal(host(got), v, equal_nan=True)      # number times scale is exact
    slots = rng.integers(-1, 5 * bs, 77).astype(np.int32)
    got = sp.unpack_fp4(dev(pool), torch_dtype(dtype), slots=dev(slots), scale=0.3)
    ref = np.where((slots < 0)[:, None, None], 0, v.reshape(-1, hk, d)[slots]) * np.float64(np.float32(0.3))
    ok = np.isnan(ref) == np.isnan(host(got))
    assert ok.all()
    near = np.abs(np.nan_to_num(host(got)) - np.nan_to_num(ref)) <= 1.001 * HALF_STEP[dtype] * np.abs(np.nan_to_num(ref)) + 2.0 ** -25
    assert near.all()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = sp.unpack_fp4(dev(pool), slots=dev(np.array([0, 5 * bs, -2], dtype=np.int32)), status=status)
    assert int(status) == 6 and not bad[1:].any()


def test_large_offsets():
    """A pool of more than 2^31 bytes."""
    import torch

    import speculative_prefill_token_gb300 as sp
    blocks, bs, d = 60000, 128, 128
    pools = [torch.zeros(blocks, 4, bs // 8, 9 * d // 2, dtype=torch.uint8, device="cuda")[:, 3:] for _ in range(2)]
    assert pools[0].stride(0) * blocks > 1 << 31
    x = torch.randn(2, 1, d, device="cuda").bfloat16()
    slots = torch.tensor([blocks * bs - 1, 5], dtype=torch.int32, device="cuda")
    sp.append_kv_fp4(x, -x, slots, *pools)
    back = [sp.unpack_fp4(p, slots=slots) for p in pools]
    codes, scales = fp4_oracle.encode(host(x).astype(np.float32))
    assert np.array_equal(host(back[0]), fp4_oracle.decode(codes, scales)) and torch.equal(back[1], -back[0])
    q = torch.randn(1, 2, d, device="cuda").bfloat16()
    table = torch.tensor([[blocks - 1]], dtype=torch.int32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    last = torch.arange((blocks - 1) * bs, blocks * bs, dtype=torch.int32, device="cuda")
    k, v = (host(sp.unpack_fp4(p, slots=last))[None] for p in pools)
    ref = paged_oracle.paged_attention(host(q), [0, 1], [bs], np.zeros((1, 1), dtype=int), k, v)
    from tests.fp4_cases import check_attention
    out = sp.paged_attention_fp4(q, i32(0, 1), i32(bs), table, *pools)
    check_attention(out, None, ref, [bs], d, "bf16", 1, 6.0)


@pytest.mark.parametrize("d,bs", [(256, 29_900_160), (64, 119_400_064)])
def test_a_block_of_more_than_32_bits(d, bs):
    """A pool of one block and one head is one run of rows: the last of them lie more than 2^32 bytes behind the first."""
    import torch

    import speculative_prefill_token_gb300 as sp
    from tests.fp4_cases import check_attention
    n, tail = 4, 70
    assert bs % 128 == 0 and (bs - tail) * (9 * d // 16) > 1 << 32
    pools = [torch.zeros(1, 1, bs // 8, 9 * d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    slots = torch.arange(bs - tail, bs, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(d)
    qkv = torch.randn(tail, 4, d, device="cuda", generator=gen).bfloat16()
    sp.append_kv_fp4(qkv[:, 2:3], qkv[:, 3:], slots, *pools)
    back = [sp.unpack_fp4(p, slots=slots) for p in pools]
    assert np.array_equal(host(back[0]), fp4_oracle.decode(*fp4_oracle.encode(host(qkv[:, 2:3]).astype(np.float32))))
    q = qkv[:n, :2].contiguous()
    ws = sp.make_attention_fp4_workspace(q, 1, pools[0], kv_tokens=0)
    out = sp.paged_attention_fp4(q, i32(0, n), i32(bs), i32(0)[None], *pools, window=60, ws=ws)
    assert sp.device_status(ws) == 0
    k, v = (host(x)[None] for x in back)
    ref = paged_oracle.paged_attention(host(q), [0, n], [tail], np.zeros((1, 1), dtype=int), k, v, window=60)
    check_attention(out, None, ref, [tail], d, "bf16", n, 6.0)


def test_a_refused_read_keeps_no_memory():
    import torch

    import speculative_prefill_token_gb300 as sp
    pool = torch.zeros(64, 2, 2, 576, dtype=torch.uint8, device="cuda")
    slots = torch.zeros(1000, dtype=torch.int64, device="cuda")
    status = torch.zeros(1, device="cuda")
    sp.unpack_fp4(pool)
    before = torch.cuda.memory_allocated()
    for kw in (dict(slots=slots), dict(status=status), dict(scale="one"), dict(scale=float("inf")), dict(slots=slots[:0].float())):
        with pytest.raises((ValueError, TypeError, sp.SpecPrefillError)):
            sp.unpack_fp4(pool, **kw)
        assert torch.cuda.memory_allocated() == before, kw
