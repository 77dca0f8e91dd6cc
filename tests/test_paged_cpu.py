"""Host-side refusals of the paged-cache operators (nothing is enqueued, so no
GPU is needed), and the oracle's own pins."""

import ctypes

import numpy as np
import pytest

import speculative_prefill_token_gb300 as sp
from oracle import paged_oracle
from speculative_prefill_token_gb300 import _build, paged

P = 1 << 20   # a 16-byte aligned address that is never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sp.load()


def _tables(lib, shape=(), **kw):
    s = dict(n_seqs=4, block_size=16, table_stride=8, n_tokens=10, free_capacity=20, pool_blocks=100)
    s.update(shape)
    a = dict(ctx_len=P, new_off=P + 64, free_blocks=P + 128, n_free=P + 192, table=P + 256, slot_map=P + 512,
             kv_len=P + 1024, n_left=P + 2048, status=None)
    a.update(kw)
    return lib.sp_block_tables(ctypes.byref(paged._BlockShape(**s)), a["ctx_len"], a["new_off"], a["free_blocks"],
                               a["n_free"], a["table"], a["slot_map"], a["kv_len"], a["n_left"], a["status"], None)


def test_block_tables_refusals(lib):
    for name in ("n_seqs", "block_size", "table_stride", "pool_blocks"):
        assert _tables(lib, {name: 0}) == 1, name
    for name in ("n_tokens", "free_capacity"):
        assert _tables(lib, {name: -1}) == 1, name
    assert _tables(lib, dict(pool_blocks=1 << 28)) == 1            # slots past 31 bits
    assert _tables(lib, dict(n_seqs=16385)) == 2
    for name in ("ctx_len", "new_off", "free_blocks", "n_free", "table", "slot_map", "kv_len", "n_left"):
        assert _tables(lib, **{name: None}) == 1, name
    # outputs on inputs or on one another
    assert _tables(lib, kv_len=P) == 1 and _tables(lib, n_left=P + 192) == 1 and _tables(lib, kv_len=P + 512) == 1
    assert _tables(lib, status=P + 2048) == 1


def _append(lib, shape=(), **kw):
    s = dict(n_tokens=4, n_q_heads=4, n_kv_heads=2, head_dim=64, rotary_dim=32, max_pos=100, dtype=0, reserved=0,
             pool_tokens=64, q_stride_token=512, q_stride_head=64, qo_stride_token=256, qo_stride_head=64,
             k_stride_token=512, k_stride_head=64, v_stride_token=512, v_stride_head=64, kp_stride_token=128,
             kp_stride_head=64, vp_stride_token=128, vp_stride_head=64)
    s.update(shape)
    names = ("q", "k", "v", "slot_map", "positions", "cos_sin", "n_new", "q_out", "k_pool", "v_pool")
    a = {n: P + 4096 * i for i, n in enumerate(names)}
    a.update(n_new=None)
    a.update(kw)
    return lib.sp_append_kv(ctypes.byref(paged._AppendShape(**s)), *[a[n] for n in names], None, None)


def test_append_kv_refusals(lib):
    for kw in (dict(n_tokens=0), dict(n_q_heads=0), dict(n_kv_heads=0), dict(head_dim=0), dict(rotary_dim=-16),
               dict(rotary_dim=80), dict(dtype=2), dict(pool_tokens=0), dict(pool_tokens=1 << 31), dict(max_pos=0),
               dict(reserved=1), dict(k_stride_token=32), dict(kp_stride_head=8)):
        assert _append(lib, kw) == 1, kw
    for kw in (dict(head_dim=72), dict(rotary_dim=24), dict(q_stride_token=516), dict(vp_stride_token=132),
               dict(head_dim=1040, rotary_dim=0)):
        assert _append(lib, kw) == 2, kw
    for name in ("k", "v", "slot_map", "positions", "cos_sin", "k_pool", "v_pool", "q", "q_out"):
        assert _append(lib, **{name: None}) == 1, name
    for name in ("q", "k", "v", "cos_sin", "q_out", "k_pool", "v_pool"):
        assert _append(lib, **{name: P + 8}) == 1, name
    assert _append(lib, k_pool=P, v_pool=P) == 1
    assert _append(lib, q=P, q_out=P) == 1       # in place with other strides


def _paged(shape=()):
    s = dict(n_seqs=2, n_q_heads=8, n_kv_heads=2, head_dim=128, dtype=0, block_size=16, table_stride=8, n_tokens=10,
             pool_tokens=256, q_stride_token=1024, q_stride_head=128, o_stride_token=1024, o_stride_head=128,
             k_stride_token=256, k_stride_head=128, v_stride_token=256, v_stride_head=128)
    s.update(shape)
    return paged._PagedShape(**s)


def _attend(lib, shape=(), params=(), ws_bytes=1 << 30, **kw):
    p = dict(causal=1, window=0, scale=0.0, spin_limit=0)
    p.update(params)
    names = ("q_off", "kv_len", "table", "q", "k_pool", "v_pool", "out", "lse", "ws")
    a = {n: P + 4096 * i for i, n in enumerate(names)}
    a.update(kw)
    return lib.sp_paged_attention(ctypes.byref(_paged(shape)), ctypes.byref(paged._AttnParams(**p)),
                                  *[a[n] for n in names], ws_bytes, None)


def test_paged_attention_refusals(lib):
    n = ctypes.c_size_t()
    for kw in (dict(n_seqs=0), dict(n_q_heads=0), dict(n_kv_heads=0), dict(table_stride=0), dict(n_tokens=0),
               dict(block_size=0), dict(pool_tokens=0), dict(pool_tokens=1 << 31), dict(n_q_heads=9), dict(dtype=2),
               dict(q_stride_token=64), dict(k_stride_head=8), dict(block_size=512)):
        assert _attend(lib, kw) == 1, kw
        assert lib.sp_paged_attention_workspace(ctypes.byref(_paged(kw)), ctypes.byref(n)) == 1, kw
    for kw in (dict(head_dim=96), dict(head_dim=512), dict(n_seqs=65537), dict(n_q_heads=258), dict(n_tokens=(1 << 30) + 1), dict(block_size=24),
               dict(block_size=192), dict(block_size=4), dict(k_stride_token=260), dict(o_stride_head=132)):
        assert _attend(lib, kw) == 2, kw
    for kw in (dict(causal=2), dict(window=-1), dict(causal=0, window=4), dict(scale=-1.0), dict(scale=float("inf")),
               dict(scale=float("nan"))):
        assert _attend(lib, params=kw) == 1, kw
    for name in ("q_off", "kv_len", "table", "q", "k_pool", "v_pool", "out"):
        assert _attend(lib, **{name: None}) == 1, name
    for name in ("q", "k_pool", "v_pool", "out"):
        assert _attend(lib, **{name: P + 8}) == 1, name
    assert _attend(lib, out=P, q=P) == 1
    assert lib.sp_paged_attention_workspace(ctypes.byref(_paged()), ctypes.byref(n)) == 0 and n.value >= 256
    assert lib.sp_paged_attention_workspace(ctypes.byref(_paged()), None) == 1
    assert _attend(lib, ws=None) == 3 and _attend(lib, ws=P + 16) == 3 and _attend(lib, ws_bytes=n.value - 1) == 3


def test_outputs_on_inputs_and_too_many_heads_are_refused(lib):
    k, v, q, k_pool, v_pool = P + 4096, P + 8192, P, P + 8 * 4096, P + 9 * 4096
    for kw in (dict(k_pool=k), dict(v_pool=v), dict(k_pool=v), dict(v_pool=q), dict(q_out=k), dict(q_out=v),
               dict(q_out=k_pool), dict(q_out=v_pool)):
        assert _append(lib, **kw) == 1, kw
    for kw in (dict(n_q_heads=(1 << 16) - 3), dict(n_kv_heads=1 << 15), dict(n_kv_heads=1 << 30), dict(n_q_heads=2 ** 31 - 1)):
        assert _append(lib, kw) == 2, kw
    assert _attend(lib, out=P + 4 * 4096) == 1 and _attend(lib, out=P + 5 * 4096) == 1
    assert _attend(lib, dict(n_q_heads=1 << 17, n_kv_heads=1 << 16)) == 2


def test_status_string_of_the_free_list(lib):
    assert lib.sp_status_string(7) == b"the free list holds too few blocks"
    assert sp.STATUS[7] == "SP_ERR_CAPACITY"


def test_binding_refuses_tensors_before_the_library():
    import torch
    t = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        sp.block_tables(t, t, t, t, t.view(3, 1), 8, n_tokens=4)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sp.append_kv(x, x, t, x, x)
    with pytest.raises(ValueError):
        sp.paged_attention(x, t, t, t, x, x)


def test_oracle_block_tables_pin():
    """Two requests, blocks of 4: the first fills its block and takes one more,
    the second starts with two; blocks come from the list's end."""
    got = paged_oracle.block_tables([3, 0], [0, 3, 8], [10, 11, 12, 13], 4, [[5, -1], [-1, -1]], 4, 9)
    assert got[0].tolist() == [[5, 13], [12, 11]]
    assert got[1].tolist() == [23, 52, 53, 48, 49, 50, 51, 44, -1]
    assert got[2].tolist() == [6, 5] and got[3] == 1
    assert paged_oracle.block_tables([3, 0], [0, 3, 8], [10, 11], 2, [[5, -1], [-1, -1]], 4, 9) is None


def test_oracle_attention_pin():
    """One head of two elements (values given), two cached tokens and one new:
    softmax of (0, log 2, log 4) over values 1, 2, 4, and the window's tail."""
    k = np.zeros((1, 8, 1, 2))
    k[0, :3, 0, 0] = [0.0, np.log(2), np.log(4)]
    v = np.zeros((1, 8, 1, 2))
    v[0, :3, 0, 1] = [1, 2, 4]
    q = np.zeros((1, 1, 2))
    q[0, 0, 0] = 1.0
    out, lse, _, _ = paged_oracle.paged_attention(q, [0, 1], [3], np.array([[0]]), k, v, scale=1.0)
    assert np.allclose(out[0, 0], [0, (1 + 4 + 16) / 7]) and np.isclose(lse[0, 0], np.log(7))
    out, lse, _, _ = paged_oracle.paged_attention(q, [0, 1], [3], np.array([[0]]), k, v, scale=1.0, window=2)
    assert np.allclose(out[0, 0, 1], (4 + 16) / 6) and np.isclose(lse[0, 0], np.log(6))


def test_oracle_rotation_pin():
    x = np.arange(6.0).reshape(1, 1, 6)
    turn = np.array([[0.0, 0.0, 1.0, 1.0]])          # a quarter turn of the first four elements
    assert paged_oracle.rotate(x, [0], turn).tolist() == [[[-2.0, -3.0, 0.0, 1.0, 4.0, 5.0]]]
