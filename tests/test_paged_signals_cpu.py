"""The bounds of long contexts can see what they are for: on the CPU, mistakes
planted in the oracle's own attention (a lost key, a lost tile of the second
product, a lost part, a key too many) are rejected, and its result in the
tensors' type is accepted."""

import numpy as np
import pytest

from oracle import paged_oracle
from tests.paged_cases import torch_dtype
from tests.paged_signals import TILE, check_signals, signal_arrays


def _attention(s, v, seen):
    """out and lse of one KV head from its logits, values and mask."""
    x = np.where(seen, s, -np.inf)
    top = x.max(-1, keepdims=True)
    p = np.exp(x - top)
    return p, p.sum(-1), p @ v, top[..., 0]


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16"), (256, "bf16")])
def test_planted_mistakes_are_rejected(d, dtype):
    import torch
    ctx, new, hq, bs = 32768, 8, 2, 16
    kv = ctx + new
    a = signal_arrays(7, [ctx], [new], hq, 1, d, bs, dtype)
    ref = paged_oracle.paged_attention(a["q"], a["q_off"], a["kv_len"], a["table"], a["k_pool"], a["v_pool"])
    pages = a["table"][0, :-(-kv // bs)]
    k = a["k_pool"][pages].reshape(-1, d)[:kv].astype(np.float64)
    v = a["v_pool"][pages].reshape(-1, d)[:kv].astype(np.float64)
    s = np.einsum("thd,kd->thk", a["q"].astype(np.float64), k) / np.sqrt(d)
    j, pos = np.arange(kv), ctx + np.arange(new)
    seen = np.broadcast_to((j <= pos[:, None])[:, None], s.shape)

    def result(num, total, top):
        out = torch.from_numpy(num / total[..., None]).to(torch_dtype(dtype))
        return out, top + np.log(total)

    def accepted(*got):
        try:
            check_signals(*got, ref, [kv], d, dtype)
        except AssertionError:
            return False
        return True

    p, total, num, top = _attention(s, v, seen)
    assert accepted(*result(num, total, top))
    tiles = -(-kv // TILE)
    # the second product without one tile, the sum intact; a part without both
    for t in (0, 1, tiles // 2, tiles - 2, tiles - 1):
        cut = slice(t * TILE, (t + 1) * TILE)
        less = num - p[..., cut] @ v[cut]
        assert not accepted(*result(less, total, top)), t
        assert not accepted(*result(less, total - p[..., cut].sum(-1), top)), t
        # 16 keys of the tile, as one step of a product takes
        cut = slice(t * TILE, t * TILE + 16)
        assert not accepted(*result(num - p[..., cut] @ v[cut], total, top)), t
        assert not accepted(*result(num - p[..., cut] @ v[cut], total - p[..., cut].sum(-1), top)), t
    # the last keys, one of them, the first one, the edges of a tile
    for lost in ([kv - 8 + i for i in range(8)], [kv - 1], [ctx - 1], [0], [TILE - 1], [TILE], [200 * TILE]):
        less = seen.copy()
        less[..., lost] = False
        _, t2, n2, m2 = _attention(s, v, less)
        assert not accepted(*result(n2, t2, m2)), lost
    # every row sees one key too many (the last one has none left)
    more = np.broadcast_to((j <= pos[:, None] + 1)[:, None], s.shape)
    _, t2, n2, m2 = _attention(s, v, more)
    assert not accepted(*result(n2, t2, m2))
    # a window of one key more or less: its edge passes the first key of a tile, a signal
    window = ctx + 1 - 200 * TILE
    ref = paged_oracle.paged_attention(a["q"], a["q_off"], a["kv_len"], a["table"], a["k_pool"], a["v_pool"],
                                       window=window)
    for w in (window - 1, window, window + 1):
        some = np.broadcast_to(((j <= pos[:, None]) & (j > pos[:, None] - w))[:, None], s.shape)
        _, t2, n2, m2 = _attention(s, v, some)
        assert accepted(*result(n2, t2, m2)) == (w == window), w
