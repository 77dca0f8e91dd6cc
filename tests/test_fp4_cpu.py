"""Host-side refusals of the 4-bit cache's and the pages' operators (nothing is
enqueued, so no GPU is needed), and the oracle's own pins."""

import ctypes

import numpy as np
import pytest

import speculative_prefill_token_gb300 as sp
from oracle import fp4_oracle
from speculative_prefill_token_gb300 import _build, fp4, pages

P = 1 << 20   # a 16-byte aligned address that is never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sp.load()


def _append(lib, shape=(), **kw):
    s = dict(n_tokens=4, n_q_heads=4, n_kv_heads=2, head_dim=64, rotary_dim=32, max_pos=100, dtype=0, block_size=16,
             pool_blocks=4, q_stride_token=512, q_stride_head=64, qo_stride_token=256, qo_stride_head=64,
             k_stride_token=512, k_stride_head=64, v_stride_token=512, v_stride_head=64, kp_stride_block=1152,
             kp_stride_head=576, vp_stride_block=1152, vp_stride_head=576, k_scale=1.0, v_scale=1.0)
    s.update(shape)
    names = ("q", "k", "v", "slot_map", "positions", "cos_sin", "n_new", "q_out", "k_pool", "v_pool")
    a = {n: P + 4096 * i for i, n in enumerate(names)}
    a.update(n_new=None, status=None)
    a.update(kw)
    return lib.sp_append_kv_fp4(ctypes.byref(fp4._AppendShape(**s)), *[a[n] for n in names], a["status"], None)


def test_append_refusals(lib):
    for kw in (dict(n_tokens=0), dict(n_q_heads=0), dict(n_kv_heads=0), dict(head_dim=0), dict(rotary_dim=-16),
               dict(rotary_dim=80), dict(dtype=2), dict(pool_blocks=0), dict(pool_blocks=1 << 27), dict(max_pos=0),
               dict(block_size=0), dict(k_stride_token=32), dict(kp_stride_head=288), dict(vp_stride_block=16),
               dict(k_scale=0.0), dict(k_scale=-1.0), dict(v_scale=float("nan")), dict(v_scale=float("inf")),
               dict(v_scale=2.0 ** -61), dict(k_scale=2.0 ** 61)):
        assert _append(lib, kw) == 1, kw
    for kw in (dict(head_dim=80), dict(head_dim=512), dict(rotary_dim=24), dict(q_stride_token=516),
               dict(block_size=24), dict(block_size=4), dict(kp_stride_block=1160), dict(vp_stride_head=584),
               dict(kp_stride_block=1 << 32), dict(n_q_heads=70000)):
        assert _append(lib, kw) == 2, kw
    for name in ("k", "v", "slot_map", "positions", "cos_sin", "k_pool", "v_pool", "q", "q_out"):
        assert _append(lib, **{name: None}) == 1, name
    for name in ("q", "k", "v", "cos_sin", "q_out", "k_pool", "v_pool"):
        assert _append(lib, **{name: P + 8}) == 1, name
    for name in ("slot_map", "positions", "n_new", "status"):
        assert _append(lib, **{name: P + 2}) == 1, name
    names = ("q", "k", "v", "slot_map", "positions", "cos_sin")
    for i, name in enumerate(names):
        assert _append(lib, k_pool=P + 4096 * i) == 1, name
        assert _append(lib, v_pool=P + 4096 * i) == 1, name
        if i:
            assert _append(lib, q_out=P + 4096 * i) == 1, name
    assert _append(lib, k_pool=P + 4096 * 9) == 1     # on v_pool
    assert _append(lib, q=P, q_out=P) == 1            # in place with other strides


def _unpack(lib, shape=(), **kw):
    s = dict(n_kv_heads=2, head_dim=64, block_size=16, dtype=0, pool_blocks=4, stride_block=1152, stride_head=576,
             n_rows=64, o_stride_token=128, o_stride_head=64, scale=1.0, reserved=0)
    s.update(shape)
    a = dict(pool=P, slots=None, out=P + 4096, status=None)
    a.update(kw)
    return lib.sp_unpack_fp4(ctypes.byref(fp4._UnpackShape(**s)), a["pool"], a["slots"], a["out"], a["status"], None)


def test_unpack_refusals(lib):
    for kw in (dict(n_rows=0), dict(n_rows=63), dict(n_kv_heads=0), dict(pool_blocks=0), dict(dtype=3), dict(reserved=1),
               dict(scale=float("nan")), dict(stride_head=64), dict(o_stride_token=32)):
        assert _unpack(lib, kw) == 1, kw
    for kw in (dict(head_dim=32), dict(block_size=12), dict(o_stride_token=132), dict(stride_block=1160)):
        assert _unpack(lib, kw) == 2, kw
    for kw in (dict(pool=None), dict(out=None), dict(out=P + 2), dict(slots=P + 1), dict(out=P), dict(status=P + 3)):
        assert _unpack(lib, **kw) == 1, kw


def _shape(shape=()):
    s = dict(n_seqs=2, n_q_heads=8, n_kv_heads=2, head_dim=128, dtype=0, block_size=16, table_stride=8, n_tokens=10,
             max_new=0, reserved=0, dense_tokens=0, pool_blocks=16, q_stride_token=1024, q_stride_head=128,
             o_stride_token=1024, o_stride_head=128, k_stride_block=2304, k_stride_head=1152, v_stride_block=2304,
             v_stride_head=1152)
    s.update(shape)
    return fp4._Shape(**s)


def _attend(lib, shape=(), params=(), ws_bytes=None, **kw):
    p = dict(causal=1, window=0, scale=0.0, k_scale=1.0, v_scale=1.0, spin_limit=0)
    p.update(params)
    names = ("q_off", "kv_len", "table", "q", "k_pool", "v_pool", "out", "lse", "ws")
    a = {n: P + 4096 * i for i, n in enumerate(names)}
    a.update(lse=None)
    a.update(kw)
    n = 1 << 40 if ws_bytes is None else ws_bytes
    return lib.sp_paged_attention_fp4(ctypes.byref(_shape(shape)), ctypes.byref(fp4._Params(**p)),
                                      *[a[x] for x in names], n, None)


def test_attention_refusals(lib):
    for kw in (dict(n_seqs=0), dict(n_q_heads=0), dict(n_kv_heads=0), dict(n_q_heads=7), dict(table_stride=0),
               dict(n_tokens=0), dict(max_new=11), dict(max_new=-1), dict(reserved=1), dict(dense_tokens=-1),
               dict(dtype=2), dict(block_size=0), dict(pool_blocks=0), dict(pool_blocks=1 << 28), dict(q_stride_token=64),
               dict(k_stride_head=64)):
        assert _attend(lib, kw) == 1, kw
    for kw in (dict(n_seqs=65537), dict(n_q_heads=512), dict(head_dim=96), dict(block_size=24), dict(q_stride_head=132),
               dict(v_stride_block=2312), dict(n_tokens=(1 << 30) + 1), dict(n_tokens=1 << 29),
               dict(dense_tokens=1 << 31), dict(k_stride_block=1 << 33)):
        assert _attend(lib, kw) == 2, kw
    for kw in (dict(causal=2), dict(window=-1), dict(causal=0, window=4), dict(scale=-1.0), dict(scale=float("nan")),
               dict(k_scale=0.0), dict(v_scale=float("inf")), dict(k_scale=2.0 ** 70), dict(scale=2.0 ** -100, k_scale=2.0 ** -60),
               dict(scale=2.0 ** 100, k_scale=2.0 ** 60)):
        assert _attend(lib, params=kw) == 1, kw
    for name in ("q_off", "kv_len", "table", "q", "k_pool", "v_pool", "out"):
        assert _attend(lib, **{name: None}) == 1, name
    names = ("q_off", "kv_len", "table", "q", "k_pool", "v_pool")
    for i, name in enumerate(names):
        assert _attend(lib, out=P + 4096 * i) == 1 and _attend(lib, lse=P + 4096 * i) == 1, name
    assert _attend(lib, lse=P + 4096 * 6) == 1 and _attend(lib, lse=P + 4096 * 8) == 1
    for name in ("q", "k_pool", "v_pool", "out"):
        assert _attend(lib, **{name: P + 4096 * 9 + 8}) == 1, name
    for name in ("q_off", "kv_len", "table", "lse"):
        assert _attend(lib, **{name: P + 4096 * 9 + 2}) == 1, name
    assert _attend(lib, ws=None) == 3 and _attend(lib, ws=P + 128) == 3 and _attend(lib, ws_bytes=4096) == 3


def test_workspace_of_the_copy(lib):
    """It grows with dense_tokens where a request can have many rows, and only there."""
    def size(**kw):
        n = ctypes.c_size_t()
        assert lib.sp_paged_attention_fp4_workspace(ctypes.byref(_shape(kw)), ctypes.byref(n)) == 0
        return n.value
    base = size()
    assert size(dense_tokens=100000) == base                     # 10 tokens x 4 heads: few rows
    many = dict(n_tokens=1000)
    grown = size(**many, dense_tokens=100000) - size(**many)
    assert grown > 100000 * 2 * 128 * 2 * 2
    assert size(**many, dense_tokens=100000, max_new=4) == size(**many, max_new=4)


def _copy(lib, shape=(), n=2, **kw):
    s = dict(n_pools=n, n_entries=4, rows=16, block_size=16, n_kv_heads=2, head_dim=64, fp4=0, n_seqs=0, table_stride=0,
             reserved=0, pool_blocks=8, stride_block=4096, stride_token=256, stride_head=128)
    s.update(shape)
    a = dict(pools=[P + (1 << 16) * i for i in range(n)], src=P + (1 << 20), dst=P + (1 << 20) + 64, table=None, off=None,
             n_used=None, status=None)
    a.update(kw)
    ptr = (ctypes.c_void_p * len(a["pools"]))(*a["pools"])
    return lib.sp_copy_kv(ctypes.byref(pages._CopyShape(**s)), ptr, a["src"], a["dst"], a["table"], a["off"], a["n_used"],
                          a["status"], None)


def test_copy_refusals(lib):
    T = P + (1 << 21)
    for kw in (dict(n_pools=0), dict(n_entries=0), dict(rows=2), dict(rows=0), dict(block_size=0), dict(n_kv_heads=0),
               dict(head_dim=0), dict(fp4=2), dict(reserved=1), dict(pool_blocks=0), dict(pool_blocks=1 << 28),
               dict(stride_token=64), dict(stride_head=16)):
        assert _copy(lib, kw) == 1, kw
    for kw in (dict(n_pools=257), dict(head_dim=68), dict(head_dim=1032), dict(stride_token=264),
               dict(fp4=1, head_dim=80), dict(fp4=1, block_size=12, rows=12), dict(n_kv_heads=70000)):
        assert _copy(lib, kw) == 2, kw
    assert _copy(lib, src=None) == 1 and _copy(lib, dst=None) == 1
    assert _copy(lib, dict(rows=1), table=T) == 1 and _copy(lib, dict(rows=1), off=T) == 1
    assert _copy(lib, dict(n_seqs=2, table_stride=4), table=T, off=T + 64) == 1            # whole blocks have no table
    assert _copy(lib, dict(rows=1, n_seqs=0, table_stride=4), table=T, off=T + 64) == 1
    assert _copy(lib, pools=[P, P]) == 1 and _copy(lib, pools=[P, None]) == 1 and _copy(lib, pools=[P, P + 8]) == 1
    assert _copy(lib, pools=[P, P + (1 << 20)]) == 1                                       # on src
    assert _copy(lib, status=P + (1 << 20)) == 1 and _copy(lib, src=P + (1 << 20) + 2) == 1


def _fork(lib, shape=(), **kw):
    s = dict(n_seqs=4, n_forks=2, block_size=16, table_stride=8, pool_blocks=20, free_capacity=20)
    s.update(shape)
    names = ("src", "dst", "ctx", "table", "shared", "free", "n_free", "kv_len", "copy_src", "copy_dst", "n_left", "status")
    a = {n: P + 4096 * i for i, n in enumerate(names)}
    a.update(status=None)
    a.update(kw)
    return lib.sp_fork_blocks(ctypes.byref(pages._PagesShape(**s)), *[a[n] for n in names], None)


def _free(lib, shape=(), **kw):
    s = dict(n_seqs=4, n_forks=0, block_size=16, table_stride=8, pool_blocks=20, free_capacity=20)
    s.update(shape)
    names = ("ctx", "new", "table", "shared", "free", "n_free", "kv_len", "n_left", "status")
    a = {n: P + 4096 * i for i, n in enumerate(names)}
    a.update(status=None)
    a.update(kw)
    return lib.sp_free_blocks(ctypes.byref(pages._PagesShape(**s)), *[a[n] for n in names], None)


def test_fork_and_free_refusals(lib):
    for kw in (dict(n_seqs=0), dict(block_size=0), dict(table_stride=0), dict(pool_blocks=0), dict(free_capacity=-1),
               dict(pool_blocks=1 << 28)):
        assert _fork(lib, kw) == 1 and _free(lib, kw) == 1, kw
    assert _fork(lib, dict(n_forks=0)) == 1
    assert _fork(lib, dict(n_forks=16385)) == 2 and _fork(lib, dict(n_seqs=16385)) == 2 and _free(lib, dict(n_seqs=16385)) == 2
    ins, outs = ("src", "dst", "ctx", "free", "n_free"), ("table", "shared", "kv_len", "copy_src", "copy_dst", "n_left")
    order = ("src", "dst", "ctx", "table", "shared", "free", "n_free", "kv_len", "copy_src", "copy_dst", "n_left")
    at = {n: P + 4096 * i for i, n in enumerate(order)}
    for o in outs + ("status",):
        for i in ins:
            assert _fork(lib, **{o: at[i]}) == 1, (o, i)
        for other in outs:
            if other != o:
                assert _fork(lib, **{o: at[other]}) == 1, (o, other)
    for n in order:
        assert _fork(lib, **{n: None}) == 1, n
        assert _fork(lib, **{n: P + 4096 * 20 + 2}) == 1, n
    ins, outs = ("ctx", "new", "table", "n_free"), ("shared", "free", "kv_len", "n_left")
    order = ("ctx", "new", "table", "shared", "free", "n_free", "kv_len", "n_left")
    at = {n: P + 4096 * i for i, n in enumerate(order)}
    for o in outs + ("status",):
        for i in ins:
            assert _free(lib, **{o: at[i]}) == 1, (o, i)
        for other in outs:
            if other != o:
                assert _free(lib, **{o: at[other]}) == 1, (o, other)
    for n in order:
        assert _free(lib, **{n: None}) == 1, n
        assert _free(lib, **{n: P + 4096 * 20 + 1}) == 1, n


def test_the_refusal_of_cuts_is_a_choice_of_frees_alone(lib):
    assert _free(lib, dict(alone=2)) == 1 and _free(lib, dict(alone=-1)) == 1
    assert _fork(lib, dict(alone=1)) == 1


def test_pool_sizes():
    pool = sp.make_pool_fp4(3, 24, 2, 128, device="cpu")
    assert pool.shape == (3, 2, 3, 576) and not pool.any()
    for args in ((3, 12, 2, 128), (3, 16, 2, 96), (3, 0, 2, 64)):
        with pytest.raises(ValueError):
            sp.make_pool_fp4(*args, device="cpu")


def test_cpu_tensors_are_refused():
    import torch
    pool = sp.make_pool_fp4(2, 16, 1, 64, device="cpu")
    with pytest.raises((ValueError, RuntimeError)):
        sp.unpack_fp4(pool)
    with pytest.raises(ValueError):
        sp.unpack_fp4(pool, torch.float32)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises((ValueError, RuntimeError)):
        sp.copy_kv([pool], i, i)
    with pytest.raises((ValueError, RuntimeError)):
        sp.copy_kv([], i, i)
    with pytest.raises((ValueError, RuntimeError)):
        sp.fork_blocks(i, i, i, i[None], i, i, i, 16)


# ------------------------------------------------------------ the oracle


def test_encode_by_hand():
    """Scale 1 (largest 6): halfway points go to the even code; scale 2 from 12; the
    smallest scale; a saturated one; a group with a NaN."""
    x = np.zeros((1, 16), dtype=np.float32)
    x[0] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6]
    want = np.array([[6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, -6]], dtype=float)
    for factor, scale in ((1.0, 56), (0.5, 64), (8.0, 32)):
        c, s = fp4_oracle.encode(x, factor)
        assert s.tolist() == [[scale]]
        assert np.array_equal(fp4_oracle.decode(c, s) * factor, want)
    tiny = np.full((1, 16), 2.0 ** -11, dtype=np.float32)
    c, s = fp4_oracle.encode(tiny)
    assert s.tolist() == [[1]] and (fp4_oracle.decode(c, s) == 0).all()   # a quarter of the smallest scale: to even
    c, s = fp4_oracle.encode(tiny * 3)
    assert (fp4_oracle.decode(c, s) == 2.0 ** -9).all()
    c, s = fp4_oracle.encode(np.full((1, 16), -1e30, dtype=np.float32))
    assert (fp4_oracle.decode(c, s) == -2688).all()
    x[0, 3] = np.nan
    c, s = fp4_oracle.encode(x)
    assert s.tolist() == [[127]] and np.isnan(fp4_oracle.decode(c, s)).all()


def test_encode_is_nearest_for_its_scale():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)).astype(np.float32)
    c, s = fp4_oracle.encode(x)
    scale = np.repeat(fp4_oracle.scale_values()[s], 16, axis=-1)
    every = np.concatenate([fp4_oracle.NUMBERS, -fp4_oracle.NUMBERS])
    best = np.abs(x[..., None] - every * scale[..., None]).min(-1)
    assert np.allclose(np.abs(x - fp4_oracle.decode(c, s)), best, rtol=1e-6, atol=1e-7)
    # the scale is within half an e4m3 step of a sixth of the largest
    top = np.abs(x.reshape(200, 4, 16)).max(-1) / 6
    assert (np.abs(fp4_oracle.scale_values()[s] - top) <= top / 16 * 1.0001).all()


def test_pack_is_undone_by_unpack():
    rng = np.random.default_rng(1)
    c = rng.integers(0, 16, (3, 24, 2, 64), dtype=np.uint8)
    s = rng.integers(0, 128, (3, 24, 2, 4), dtype=np.uint8)
    pool = fp4_oracle.pack(c, s)
    assert pool.shape == (3, 2, 3, 288)
    # token 10 of block 1, head 1: row 2 of record 1
    assert pool[1, 1, 1, 2 * 32] == c[1, 10, 1, 0] + 16 * c[1, 10, 1, 1] and pool[1, 1, 1, 256 + 2 * 4 + 3] == s[1, 10, 1, 3]
    back = fp4_oracle.unpack(pool)
    assert np.array_equal(back[0], c) and np.array_equal(back[1], s)


def test_forks_and_frees_by_hand():
    table = np.array([[7, 3, 5], [-1, -1, -1], [-1, -1, -1]])
    kv, cs, cd, left, t, sh = fp4_oracle.fork_blocks([0, 0], [2, 1], [10, 0, 0], table, np.zeros(8, int), [0, 1, 2], 3, 4)
    assert kv.tolist() == [10, 10, 10] and left == 1
    assert cs.tolist() == [5, 5] and cd.tolist() == [2, 1]
    assert t.tolist() == [[7, 3, 5], [7, 3, 1], [7, 3, 2]] and sh.tolist() == [0, 0, 0, 2, 0, 0, 0, 2]
    kv, n, sh2, free = fp4_oracle.free_blocks(kv, [0, 10, 5], t, sh, [0, 9, 9, 9], 1, 4)
    assert n == 3 and free.tolist() == [0, 2, 5, 9]     # the fork's begun block (cut) and the parent's
    assert sh2.tolist() == [0, 0, 0, 1, 0, 0, 0, 1]
    assert fp4_oracle.free_blocks([4, 4], [0, 0], np.array([[1], [1]]), np.zeros(4, int), [0], 0, 4) is None
