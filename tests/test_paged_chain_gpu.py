"""Steps of block_tables chained on the device, one of which cannot be served."""

import numpy as np
import pytest

from oracle import paged_oracle
from tests.paged_cases import host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("short", ["free", "row"])
def test_a_step_that_is_not_served_leaves_the_chain_as_it_was(cuda_lib, captured, short):
    """Decode steps whose lengths move on where status is 0: from the step on
    that runs out of blocks (or out of its table row) nothing changes; with
    blocks given (or the request set back) and status cleared they go on."""
    import torch
    sp = cuda_lib
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    bs, ctx, batch = 4, [6, 0, 9], 3
    ids = np.random.default_rng(0).permutation(40)
    table = np.full((batch, 5), -9)
    table[0, :2], table[2, :3] = ids[:2], ids[2:5]
    free = ids[5:].copy()
    n_free = 4 if short == "free" else 30
    if short == "row":
        table = table[:, :4]   # request 2 has room for 16 tokens
    off = np.arange(batch + 1)
    s = dict(ctx=i32(ctx), off=i32(off), free=i32(free), n_free=i32([n_free]), table=i32(table), slots=i32([0] * batch),
             kv=i32([0] * batch), left=i32([0]), status=i32([0]))

    def step():
        sp.block_tables(s["ctx"], s["off"], s["free"], s["n_free"], s["table"], bs, slot_map=s["slots"], kv_len=s["kv"],
                        n_left=s["left"], status=s["status"])
        s["ctx"].copy_(torch.where(s["status"] == 0, s["kv"], s["ctx"]))
        s["n_free"].copy_(torch.where(s["status"] == 0, s["left"], s["n_free"]))

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        step = graph.replay
    want = (table, None, np.asarray(ctx), n_free)
    served = 0
    for _ in range(12):
        step()
        now = paged_oracle.block_tables(want[2], off, free, want[3], want[0], bs, batch) if short == "free" or max(
            want[2]) < 16 else None
        if now is None:
            break
        served += 1
        want = now
        assert int(s["status"]) == 0 and np.array_equal(host(s["slots"]), want[1])
    assert served >= 5

    def unchanged():
        return (np.array_equal(host(s["table"]), want[0]) and np.array_equal(host(s["ctx"]), want[2])
                and int(s["n_free"]) == want[3])

    for _ in range(3):
        assert int(s["status"]) == (7 if short == "free" else 6) and unchanged() and (host(s["slots"]) == -1).all()
        step()
    # the caller helps, and clears the status
    if short == "free":
        free[:30] = free[4:34]   # (the four before are taken)
        s["free"].copy_(i32(free))
        s["n_free"].fill_(30)
        want = (want[0], None, want[2], 30)
    else:
        s["ctx"][2] = 2
        want = (want[0], None, np.where(np.arange(3) == 2, 2, want[2]), want[3])
    s["status"].zero_()
    for _ in range(2):
        step()
        want = paged_oracle.block_tables(want[2], off, free, want[3], want[0], bs, batch)
        assert int(s["status"]) == 0 and unchanged() and np.array_equal(host(s["slots"]), want[1])


def test_bounds_that_bound_nothing_are_refused(cuda_lib):
    """pool_blocks and n_tokens below their range are errors, not 'no bound'."""
    import torch
    sp = cuda_lib
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (i32(0), i32(0, 2), i32(0, 1), i32(2), i32(-1, -1)[None], 4)
    for kw in (dict(pool_blocks=0), dict(pool_blocks=-1), dict(n_tokens=-1)):
        slots = i32(5, 5)
        with pytest.raises(sp.SpecPrefillError):
            sp.block_tables(*args, slot_map=slots, **kw)
        assert slots.tolist() == [5, 5]
    assert sp.block_tables(*args, slot_map=i32(5, 5), pool_blocks=2)[0].tolist() == [4, 5]
    assert sp.block_tables(*args, slot_map=i32(5, 5, 5), n_tokens=2)[0].tolist() == [4, 5, 5]
