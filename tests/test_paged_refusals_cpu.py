"""Refusals of the paged-cache operators that the C ABI promises for every
output (nothing is enqueued, so no GPU is needed)."""

import pytest

from tests.test_paged_cpu import P, _append, _attend, _tables, lib  # noqa: F401  (lib is a fixture)


def test_lse_on_an_input_or_on_out_is_refused(lib):  # noqa: F811
    names = ("q_off", "kv_len", "table", "q", "k_pool", "v_pool", "out")
    for i, name in enumerate(names):
        assert _attend(lib, lse=P + 4096 * i) == 1, name
    for i, name in enumerate(names[:3]):
        assert _attend(lib, out=P + 4096 * i) == 1, name
    assert _attend(lib, ws=P + 4096 * 7) == 1   # the workspace on lse


def test_append_kv_outputs_on_index_tensors_are_refused(lib):  # noqa: F811
    names = ("q", "k", "v", "slot_map", "positions", "cos_sin")
    for i, name in enumerate(names):
        assert _append(lib, k_pool=P + 4096 * i) == 1, name
        assert _append(lib, v_pool=P + 4096 * i) == 1, name
        if i:
            assert _append(lib, q_out=P + 4096 * i) == 1, name


@pytest.mark.parametrize("by", [1, 2, 3])
def test_entries_off_their_alignment_are_refused(lib, by):  # noqa: F811
    for i, name in enumerate(("q_off", "kv_len", "table")):
        assert _attend(lib, **{name: P + 4096 * i + by}) == 1, name
    assert _attend(lib, lse=P + 4096 * 7 + by) == 1
    for name, at in dict(ctx_len=0, new_off=64, free_blocks=128, n_free=192, table=256, slot_map=512, kv_len=1024,
                         n_left=2048).items():
        assert _tables(lib, **{name: P + at + by}) == 1, name
    assert _tables(lib, status=P + 4096 + by) == 1
    for i, name in ((3, "slot_map"), (4, "positions"), (6, "n_new")):
        assert _append(lib, **{name: P + 4096 * i + by}) == 1, name
