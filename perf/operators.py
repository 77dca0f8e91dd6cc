"""The sparse-prefill operators over a block-paged cache, as cases to measure.

After the selection the target model prefills the kept tokens and then decodes.
Three operators carry that on a block-paged cache:

  tables     block tables and slot map of a step, built on the GPU from the
             requests' lengths (the kept counts are known on the device only)
  append     queries and keys rotated to their original positions, keys and
             values stored at the step's slots
  attention  attention of a chunk of new tokens (or of single tokens) over the
             paged cache

``run`` computes them in elementary torch operations, or through the library
where ``own`` is set. Head layouts and lengths are those of the repository's
workloads (8/2 heads of 256 and 16/4 of 128 with 32K to 131K prompts, 16 ragged
prompts of 4K to 16K, 4/2 heads of 64) or generic ones.
"""

import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # block tables of one decode step of the 16-prompt serving batch
        dict(name="tables_decode", kind="tables", batch=16, ctx_lo=4096, ctx_hi=16384, new_lo=1, new_hi=1,
             singles=1.0, empty=0.0, block=16, lens=1),
        # block tables of a sparse prefill: what selection keeps of 16 prompts, new requests
        dict(name="tables_prefill", kind="tables", batch=16, ctx_lo=0, ctx_hi=0, new_lo=1229, new_hi=4915,
             singles=0.0, empty=0.0, block=64, lens=2),
        # block tables of a large pool of requests, most of them decoding, some idle, some with a chunk
        dict(name="tables_many", kind="tables", batch=4000, ctx_lo=0, ctx_hi=8192, new_lo=2, new_hi=500,
             singles=0.7, empty=0.1, block=32, lens=3),
        # the new tokens of a decode step of 16 requests: rotate and store
        dict(name="append_decode", kind="append", tokens=16, hq=8, hk=2, d=256, rotary=64, dtype="bf16",
             block=16, max_pos=32768),
        # the kept tokens of the 131K-token prompt (30 %) in one layer: rotate and store
        dict(name="append_long", kind="append", tokens=39322, hq=16, hk=4, d=128, rotary=128, dtype="bf16",
             block=64, max_pos=131072),
        # one token of one short request: latency
        dict(name="attn_one", kind="attention", dtype="bf16", hq=4, hk=2, d=64, block=16, batch=1, ctx_lo=511,
             ctx_hi=511, new_lo=1, new_hi=1, singles=1.0, empty=0.0, causal=True, window=0, lens=4),
        # a decode step of the serving batch, ragged contexts, small pages
        dict(name="attn_decode_serving", kind="attention", dtype="bf16", hq=8, hk=2, d=256, block=16, batch=16,
             ctx_lo=4096, ctx_hi=16384, new_lo=1, new_hi=1, singles=1.0, empty=0.0, causal=True, window=0, lens=5),
        # a decode step of 64 requests with long contexts
        dict(name="attn_decode_long", kind="attention", dtype="bf16", hq=16, hk=4, d=128, block=64, batch=64,
             ctx_lo=2048, ctx_hi=32767, new_lo=1, new_hi=1, singles=1.0, empty=0.0, causal=True, window=0, lens=6),
        # the draft's 8 lookahead tokens after a 32K prompt
        dict(name="attn_lookahead", kind="attention", dtype="bf16", hq=8, hk=2, d=256, block=16, batch=1,
             ctx_lo=32768, ctx_hi=32768, new_lo=8, new_hi=8, singles=0.0, empty=0.0, causal=True, window=0, lens=7),
        # sparse prefill of the 32K prompt at 15 %: a new request
        dict(name="attn_prefill", kind="attention", dtype="bf16", hq=8, hk=2, d=256, block=64, batch=1,
             ctx_lo=0, ctx_hi=0, new_lo=4916, new_hi=4916, singles=0.0, empty=0.0, causal=True, window=0, lens=8),
        # the last chunk of the sparse prefill of the 131K prompt at 30 %
        dict(name="attn_chunk_long", kind="attention", dtype="bf16", hq=16, hk=4, d=128, block=64, batch=1,
             ctx_lo=35226, ctx_hi=35226, new_lo=4096, new_hi=4096, singles=0.0, empty=0.0, causal=True, window=0,
             lens=9),
        # decode steps and ragged chunks in one batch, an odd group, a sliding window, idle requests
        dict(name="attn_mixed", kind="attention", dtype="fp16", hq=15, hk=3, d=64, block=32, batch=24,
             ctx_lo=1, ctx_hi=6000, new_lo=2, new_hi=700, singles=0.5, empty=0.1, causal=True, window=1500, lens=10),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["tables", "append", "attention", "attention", "attention"])
    block = rng.choice([8, 16, 32, 64, 128, 256])
    if kind == "tables":
        batch = _log_int(rng, 1, 4000)
        new_hi = _log_int(rng, 1, max(1, min(8192, 400000 // batch)))
        ctx_hi = _log_int(rng, 1, 8192)
        return dict(kind=kind, batch=batch, ctx_lo=rng.choice([0, ctx_hi // 2]), ctx_hi=ctx_hi, new_lo=(new_hi + 1) // 2,
                    new_hi=new_hi, singles=round(rng.random(), 2), empty=rng.choice([0.0, 0.1, 0.3]), block=block,
                    lens=rng.randrange(1 << 20))
    d = rng.choice([64, 128, 256])
    hk = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if kind == "append":
        most = max(1, 39322 * 24 * 128 // ((hk * group + 2 * hk) * d))
        return dict(kind=kind, tokens=_log_int(rng, 1, min(39322, most)), hq=hk * group, hk=hk, d=d,
                    rotary=rng.choice([0, d // 4, d // 2, d]), dtype=dtype, block=block,
                    max_pos=_log_int(rng, 40000, 200000))
    form = rng.choice(["decode", "chunk", "prefill", "mixed"])
    case = dict(kind=kind, dtype=dtype, hq=hk * group, hk=hk, d=d, block=block, causal=rng.random() < 0.85, window=0,
                singles=0.0, empty=0.0, lens=rng.randrange(1 << 20))
    if form == "decode":
        batch, ctx_hi = _log_int(rng, 1, 64), _log_int(rng, 16, 32767)
        # at most the keys of the largest listed case, here and below
        ctx_hi = max(1, min(ctx_hi, 64 * 16384 * 4 * 128 // (batch * hk * d)))
        case.update(batch=batch, ctx_lo=(ctx_hi + 1) // 2, ctx_hi=ctx_hi, new_lo=1, new_hi=1, singles=1.0,
                    empty=rng.choice([0.0, 0.1]))
    elif form == "chunk":
        new, ctx = _log_int(rng, 2, 1200), _log_int(rng, 1, 20000)
        case.update(batch=1, ctx_lo=ctx, ctx_hi=ctx, new_lo=new, new_hi=new)
    elif form == "prefill":
        new = _log_int(rng, 1, 4000)
        case.update(batch=1, ctx_lo=0, ctx_hi=0, new_lo=new, new_hi=new)
    else:
        case.update(batch=rng.randrange(2, 25), ctx_lo=rng.choice([0, 1]), ctx_hi=_log_int(rng, 30, 4000), new_lo=2,
                    new_hi=_log_int(rng, 3, 500), singles=round(rng.random(), 2), empty=rng.choice([0.0, 0.2]))
    if case["causal"] and rng.random() < 0.3:
        case["window"] = _log_int(rng, 1, 4096)
    return case


def _lengths(case):
    """(cached tokens, new tokens) of every request: plain values of the case."""
    rng = random.Random(case["lens"])
    ctx, new = [], []
    for _ in range(case["batch"]):
        ctx.append(rng.randint(case["ctx_lo"], case["ctx_hi"]))
        u = rng.random()
        idle = rng.random() < case["empty"]
        new.append(0 if idle else 1 if u < case["singles"] else rng.randint(case["new_lo"], case["new_hi"]))
    if sum(new) == 0:
        new[0] = 1
    return ctx, new


def _offsets(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return off


def _blocks(n, block):
    return -(-n // block)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_tables(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ctx, new = _lengths(case)
    bs = case["block"]
    held = [_blocks(c, bs) for c in ctx]
    need = [_blocks(c + n, bs) for c, n in zip(ctx, new)]
    taken = sum(n - h for n, h in zip(need, held))
    spare = taken // 8 + 5
    ids = torch.randperm(sum(held) + taken + spare, generator=gen, device="cuda").to(torch.int32)
    width = max(max(need), 1) + 3
    # the blocks that the requests hold already; the other entries are stale
    col = torch.arange(width, device="cuda")
    first = torch.tensor(_offsets(held)[:-1], device="cuda")
    index = (first[:, None] + col).clamp(max=ids.numel() - 1)
    table = torch.where(col < torch.tensor(held, device="cuda")[:, None], ids[index], -7).to(torch.int32)
    free = ids[sum(held):].contiguous()
    tokens = sum(new)
    return dict(kind="tables", block=bs, tokens=tokens, ctx_len=_i32(ctx), new_off=_i32(_offsets(new)), free=free,
                n_free=_i32([free.numel()]), table=table.contiguous(),
                # a step's buffers hold a few rows more than it has tokens
                slot_map=torch.zeros(tokens + 5, dtype=torch.int32, device="cuda"),
                kv_len=torch.zeros(len(ctx), dtype=torch.int32, device="cuda"),
                n_left=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _plain_tables(s):
    bs, rows = s["block"], s["slot_map"].numel()
    ctx = s["ctx_len"].long()
    off = s["new_off"].long()
    new = off[1:] - off[:-1]
    held, need = (ctx + bs - 1) // bs, (ctx + new + bs - 1) // bs
    take = need - held
    before = torch.cumsum(take, 0) - take
    n_free = s["n_free"].long()
    # table entries [held, need) of each request: the free list from its end
    col = torch.arange(s["table"].shape[1], device="cuda")
    index = (n_free - 1 - (before[:, None] + col - held[:, None])).clamp(0, s["free"].numel() - 1)
    fresh = (col >= held[:, None]) & (col < need[:, None])
    s["table"].copy_(torch.where(fresh, s["free"][index], s["table"]))
    # a slot for each new token, -1 behind the last
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(off[1:], t, right=True).clamp(max=ctx.numel() - 1)
    pos = ctx[b] + t - off[b]
    k = (pos // bs).clamp(0, s["table"].shape[1] - 1)
    slot = s["table"][b, k].long() * bs + pos % bs
    s["slot_map"].copy_(torch.where(t < off[-1], slot, -1))
    s["kv_len"].copy_(ctx + new)
    s["n_left"].copy_(n_free - take.sum())
    return s["table"], s["slot_map"], s["kv_len"], s["n_left"]


def _prepare_append(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, hq, hk, d, bs, rot = (case[x] for x in ("tokens", "hq", "hk", "d", "block", "rotary"))
    dtype = _TYPES[case["dtype"]]
    # one row of queries, keys and values for each token, as a projection leaves it
    qkv = torch.randn(n, hq + 2 * hk, d, generator=gen, device="cuda").to(dtype)
    blocks = _blocks(n, bs) + 3
    perm = torch.randperm(blocks, generator=gen, device="cuda")
    t = torch.arange(n, device="cuda")
    slots = (perm[t // bs] * bs + t % bs).to(torch.int32)
    # original positions of the kept tokens, increasing
    positions = torch.randperm(case["max_pos"], generator=gen, device="cuda")[:n].sort().values.to(torch.int32)
    table = None
    if rot:
        inv = 1.0e7 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") * 2.0 / rot)
        angle = torch.arange(case["max_pos"], dtype=torch.float64, device="cuda")[:, None] * inv
        table = torch.cat([angle.cos(), angle.sin()], 1).float()
    pools = [torch.randn(blocks, bs, hk, d, generator=gen, device="cuda").to(dtype) for _ in range(2)]
    return dict(kind="append", rotary=rot, q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], slots=slots,
                positions=positions, cos_sin=table, k_pool=pools[0], v_pool=pools[1],
                q_out=torch.zeros(n, hq, d, dtype=dtype, device="cuda"))


def _plain_append(s):
    half = s["rotary"] // 2

    def rotated(x):
        if not half:
            return x
        x = x.float()
        angle = s["cos_sin"][s["positions"].long()][:, None]
        cos, sin = angle[..., :half], angle[..., half:]
        a, b = x[..., :half], x[..., half:2 * half]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]], -1)

    at = s["slots"].long()
    dtype = s["q"].dtype
    s["q_out"].copy_(rotated(s["q"]))
    s["k_pool"].flatten(0, 1)[at] = rotated(s["k"]).to(dtype)
    s["v_pool"].flatten(0, 1)[at] = s["v"]
    return s["q_out"], s["k_pool"], s["v_pool"]


def _prepare_attention(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hq, hk, d, bs = (case[x] for x in ("hq", "hk", "d", "block"))
    dtype = _TYPES[case["dtype"]]
    ctx, new = _lengths(case)
    kv = [c + n for c, n in zip(ctx, new)]
    used = [_blocks(n, bs) for n in kv]
    blocks = sum(used) + 3
    perm = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    width = max(max(used), 1)
    col = torch.arange(width, device="cuda")
    first = torch.tensor(_offsets(used)[:-1], device="cuda")
    table = torch.where(col < torch.tensor(used, device="cuda")[:, None],
                        perm[(first[:, None] + col).clamp(max=blocks - 1)], 0).to(torch.int32).contiguous()
    # normalised queries and keys, a share of every head common to all tokens, and
    # first tokens that point along it: attention with sinks and a long tail
    along = torch.randn(hk, d, generator=gen, device="cuda")
    along = along / along.norm(dim=1, keepdim=True) * d ** 0.5
    k = torch.randn(blocks, bs, hk, d, generator=gen, device="cuda", dtype=torch.float32)
    begin = torch.tensor([i for i, n in enumerate(used) if n], device="cuda")
    k[table[begin, 0].long(), 0] = along * 0.8
    v = torch.randn(blocks, bs, hk, d, generator=gen, device="cuda", dtype=torch.float32)
    tokens = sum(new)
    q = torch.randn(tokens, hk, hq // hk, d, generator=gen, device="cuda", dtype=torch.float32) * 1.5
    q = (q + 0.5 * along[:, None]).reshape(tokens, hq, d)
    s = dict(kind="attention", causal=case["causal"], window=case["window"], tokens=tokens, max_new=max(new),
             max_kv=max(kv), q=q.to(dtype), k_pool=k.to(dtype), v_pool=v.to(dtype), table=table, kv_len=_i32(kv),
             q_off=_i32(_offsets(new)), out=torch.zeros(tokens, hq, d, dtype=dtype, device="cuda"),
             lse=torch.zeros(tokens, hq, dtype=torch.float32, device="cuda"), ws=None)
    if own:
        import speculative_prefill_token_gb300 as sp
        s["ws"] = sp.make_attention_workspace(s["q"], len(new), s["k_pool"])
    return s


def _plain_attention(s):
    q, table, bs = s["q"], s["table"], s["k_pool"].shape[1]
    tokens, hq, d = q.shape
    hk = s["k_pool"].shape[2]
    g = hq // hk
    off, kv = s["q_off"].long(), s["kv_len"].long()
    new = off[1:] - off[:-1]
    batch = kv.numel()
    # the cached rows of every request, [B, Hk, keys, d]; zeros behind its end
    j = torch.arange(s["max_kv"], device="cuda")
    there = j < kv[:, None]
    rows = torch.where(there, table[:, j // bs].long() * bs + j % bs, 0)
    keys = s["k_pool"].flatten(0, 1)[rows].float().masked_fill(~there[..., None, None], 0.0).transpose(1, 2)
    values = s["v_pool"].flatten(0, 1)[rows].float().masked_fill(~there[..., None, None], 0.0).transpose(1, 2)
    # the new tokens of every request, [B, Hk, G * new, d]
    i = torch.arange(s["max_new"], device="cuda")
    index = (off[:-1, None] + i).clamp(max=tokens - 1)
    qs = q[index].float().view(batch, -1, hk, g, d).permute(0, 2, 3, 1, 4).reshape(batch, hk, -1, d)
    scores = torch.matmul(qs, keys.transpose(2, 3)).view(batch, hk, g, -1, s["max_kv"]) * d ** -0.5
    seen = there[:, None, :].expand(batch, s["max_new"], -1)
    if s["causal"]:
        pos = (kv - new)[:, None] + i
        seen = seen & (j <= pos[..., None])
        if s["window"]:
            seen = seen & (j > pos[..., None] - s["window"])
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(batch, hk, -1, s["max_kv"]), values).view(batch, hk, g, -1, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (torch.log(total) + top)[..., 0]
    t = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(off[1:], t, right=True).clamp(max=batch - 1)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4)[b, t - off[b]].reshape(tokens, hq, d))
    s["lse"].copy_(lse.permute(0, 3, 1, 2)[b, t - off[b]].reshape(tokens, hq))
    return s["out"], s["lse"]


def prepare(case, seed):
    if case["kind"] == "tables":
        return _prepare_tables(case, seed)
    if case["kind"] == "append":
        return _prepare_append(case, seed)
    return _prepare_attention(case, seed)


def run(s):
    if own:
        import speculative_prefill_token_gb300 as sp
        if s["kind"] == "tables":
            sp.block_tables(s["ctx_len"], s["new_off"], s["free"], s["n_free"], s["table"], s["block"],
                            slot_map=s["slot_map"], kv_len=s["kv_len"], n_left=s["n_left"])
            return s["table"], s["slot_map"], s["kv_len"], s["n_left"]
        if s["kind"] == "append":
            sp.append_kv(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], q=s["q"], q_out=s["q_out"],
                         positions=s["positions"] if s["rotary"] else None, cos_sin=s["cos_sin"])
            return s["q_out"], s["k_pool"], s["v_pool"]
        sp.paged_attention(s["q"], s["q_off"], s["kv_len"], s["table"], s["k_pool"], s["v_pool"], causal=s["causal"],
                           window=s["window"], out=s["out"], lse=s["lse"], ws=s["ws"])
        return s["out"], s["lse"]
    if s["kind"] == "tables":
        return _plain_tables(s)
    if s["kind"] == "append":
        return _plain_append(s)
    return _plain_attention(s)


def _pairs(case, ctx, new):
    """(query, key) pairs that the masks leave, and keys that some query sees."""
    pairs = keys = 0
    for c, n in zip(ctx, new):
        if n == 0:
            continue
        if not case["causal"]:
            pairs += n * (c + n)
            keys += c + n
        else:
            w = case["window"] or c + n
            full = max(0, min(n, w - c))  # queries that see every key up to their own
            pairs += sum((c * full + full * (full + 1) // 2, (n - full) * w))
            keys += min(c + n, n - 1 + w)
    return pairs, keys


def work(case):
    if case["kind"] == "append":
        n, hq, hk, d = case["tokens"], case["hq"], case["hk"], case["d"]
        rows = n * (hq + 2 * hk)
        return {"bytes": 2 * rows * d * 2 + n * (8 + 4 * case["rotary"]), "flops": 3 * n * (hq + hk) * case["rotary"]}
    ctx, new = _lengths(case)
    if case["kind"] == "tables":
        bs = case["block"]
        taken = sum(_blocks(c + n, bs) - _blocks(c, bs) for c, n in zip(ctx, new))
        part = sum(1 for c, n in zip(ctx, new) if n and c % bs)
        return {"bytes": 4 * (3 * len(ctx) + 1 + 2 * taken + part + sum(new) + 5 + 2), "flops": 0}
    pairs, keys = _pairs(case, ctx, new)
    hq, hk, d = case["hq"], case["hk"], case["d"]
    table = sum(_blocks(c + n, case["block"]) for c, n in zip(ctx, new))
    return {"bytes": 2 * 2 * keys * hk * d + 2 * 2 * sum(new) * hq * d + 4 * sum(new) * hq + 4 * table + 8 * len(ctx),
            "flops": 4 * d * hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "tables":
        ctx, new = _lengths(case)
        bs = case["block"]
        free = s["free"].tolist()
        table = s["table"].tolist()
        slots = []
        for b, (c, n) in enumerate(zip(ctx, new)):
            for p in range(c, c + n):
                if p % bs == 0:
                    table[b][p // bs] = free.pop()
                slots.append(table[b][p // bs] * bs + p % bs)
        slots += [-1] * (s["slot_map"].numel() - len(slots))
        return (torch.tensor(table), torch.tensor(slots), torch.tensor([c + n for c, n in zip(ctx, new)]),
                torch.tensor([len(free)]))
    if case["kind"] == "append":
        r = case["rotary"] // 2
        out = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            if r:
                z = torch.complex(y[..., :r], y[..., r:2 * r])
                turn = s["cos_sin"].double()[s["positions"].long()]
                z = z * torch.complex(turn[:, :r], turn[:, r:])[:, None]
                y[..., :r], y[..., r:2 * r] = z.real, z.imag
            out.append(y)
        pools = []
        for pool, rows in ((s["k_pool"], out[1]), (s["v_pool"], s["v"].double())):
            whole = pool.double().view(-1, case["hk"], case["d"])
            whole[s["slots"].long()] = rows
            pools.append(whole.view(pool.shape))
        return out[0], pools[0], pools[1]
    ctx, new = _lengths(case)
    hq, hk, d, bs = (case[x] for x in ("hq", "hk", "d", "block"))
    g = hq // hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    first = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        pages = s["table"][b, :_blocks(c + n, bs)].long()
        for h in range(hk):
            k = s["k_pool"][pages, :, h].reshape(-1, d)[:c + n].double()
            v = s["v_pool"][pages, :, h].reshape(-1, d)[:c + n].double()
            for at in range(0, n, 512):
                m = min(512, n - at)
                q = s["q"][first + at:first + at + m, h * g:(h + 1) * g].double()
                x = torch.einsum("tgd,kd->tgk", q, k) / math.sqrt(d)
                if case["causal"]:
                    gap = (torch.arange(c + at, c + at + m, device="cuda")[:, None]
                           - torch.arange(c + n, device="cuda"))
                    hide = gap < 0
                    if case["window"]:
                        hide |= gap >= case["window"]
                    x.masked_fill_(hide[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[first + at:first + at + m, h * g:(h + 1) * g] = z
                out[first + at:first + at + m, h * g:(h + 1) * g] = torch.einsum("tgk,kd->tgd", torch.exp(x - z[..., None]), v)
        first += n
    return out, lse
