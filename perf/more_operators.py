"""The operators of a 4-bit block-paged cache and of its pages, as cases to measure.

A cache in 4 bits holds four times the context of a 16-bit one, and a decode
step reads a quarter of the bytes. An element is an e2m1 number (0, 0.5, 1,
1.5, 2, 3, 4, 6 and their negatives), sixteen neighbours of a head share an e4m3
scale, and a pool one factor. A pool is ``uint8 [blocks, Hk, block_size / 8,
9 d / 2]``: for eight tokens of a head their codes (d / 2 bytes each, the even
element in the low four bits), then their scales (d / 16 bytes each).

  append     queries and keys rotated, keys and values stored in 4 bits; the
             pools come back as the values that they stand for
  attention  attention of a chunk of new tokens (or of single tokens) over the
             4-bit cache
  copy       rows or whole blocks of the cache copied in every pool: the begun
             blocks of forked requests, and the kept tokens of a cached prompt
  pages      requests forked (full blocks shared, begun blocks taken anew), and
             the forks freed again

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
_GROUP = 16                    # elements that share a scale
_MOST = 6.0                    # largest e2m1 number
_LEAST_SCALE = 2.0 ** -9       # smallest e4m3 number above zero
_NUMBERS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    attn = dict(kind="attention", causal=True, window=0, k_scale=1.0, v_scale=1.0)
    return [
        # the new tokens of a decode step of 16 requests: rotate and store
        dict(name="append4_decode", kind="append", tokens=16, hq=8, hk=2, d=256, rotary=64, dtype="bf16", block=16,
             max_pos=32768, k_scale=1.0, v_scale=1.0),
        # the kept tokens of the 131K-token prompt (30 %) in one layer: rotate and store
        dict(name="append4_long", kind="append", tokens=39322, hq=16, hk=4, d=128, rotary=128, dtype="bf16", block=64,
             max_pos=131072, k_scale=1.0, v_scale=0.25),
        # one token of one short request: latency
        dict(attn, name="attn4_one", dtype="bf16", hq=4, hk=2, d=64, block=16, batch=1, ctx_lo=511, ctx_hi=511,
             new_lo=1, new_hi=1, singles=1.0, empty=0.0, lens=4),
        # a decode step of the serving batch, ragged contexts, small pages
        dict(attn, name="attn4_decode_serving", dtype="bf16", hq=8, hk=2, d=256, block=16, batch=16, ctx_lo=4096,
             ctx_hi=16384, new_lo=1, new_hi=1, singles=1.0, empty=0.0, lens=5),
        # a decode step of 64 requests with long contexts
        dict(attn, name="attn4_decode_long", dtype="bf16", hq=16, hk=4, d=128, block=64, batch=64, ctx_lo=2048,
             ctx_hi=32767, new_lo=1, new_hi=1, singles=1.0, empty=0.0, lens=6),
        # the draft's 8 lookahead tokens after a 32K prompt
        dict(attn, name="attn4_lookahead", dtype="bf16", hq=8, hk=2, d=256, block=16, batch=1, ctx_lo=32768,
             ctx_hi=32768, new_lo=8, new_hi=8, singles=0.0, empty=0.0, lens=7),
        # the last chunk of the sparse prefill of the 131K prompt at 30 %
        dict(attn, name="attn4_chunk_long", dtype="bf16", hq=16, hk=4, d=128, block=64, batch=1, ctx_lo=35226,
             ctx_hi=35226, new_lo=4096, new_hi=4096, singles=0.0, empty=0.0, lens=9),
        # decode steps and ragged chunks in one batch, an odd group, a sliding window, idle requests
        dict(attn, name="attn4_mixed", dtype="fp16", hq=15, hk=3, d=64, block=32, batch=24, ctx_lo=1, ctx_hi=6000,
             new_lo=2, new_hi=700, singles=0.5, empty=0.1, window=1500, k_scale=0.5, v_scale=0.125, lens=10),
        # the begun blocks of 16 forks, in the key and value pools of 6 layers
        dict(name="copy_fork", kind="copy", form="blocks", entries=16, idle=0.2, layers=6, hk=2, d=256, block=64,
             dtype="bf16", tokens=16384),
        # the kept tokens (30 %) of a cached prompt of 131K tokens moved to blocks of their own, one layer
        dict(name="copy_compact", kind="copy", form="tokens", entries=39322, idle=0.0, layers=1, hk=4, d=128, block=64,
             dtype="bf16", tokens=131072),
        # four continuations of a 32K prompt
        dict(name="pages_few", kind="pages", parents=1, forks=4, ctx_lo=32768 - 5, ctx_hi=32768, block=16, idle=0.0,
             lens=11),
        # eight continuations of each of 400 requests, some of them idle
        dict(name="pages_many", kind="pages", parents=400, forks=8, ctx_lo=0, ctx_hi=8192, block=32, idle=0.1, lens=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "attention", "attention", "attention", "copy", "pages"])
    block = rng.choice([8, 16, 32, 64, 128, 256])
    if kind == "pages":
        parents = _log_int(rng, 1, 400)
        forks = _log_int(rng, 1, min(64, 3200 // parents))
        # at most the table entries of the largest listed case
        most = 400 * 8 * 4096 // 32 * block // (parents * forks)
        ctx_hi = min(_log_int(rng, 1, 32768), max(1, most))
        return dict(kind=kind, parents=parents, forks=forks, ctx_lo=rng.choice([0, ctx_hi // 2]), ctx_hi=ctx_hi,
                    block=block, idle=rng.choice([0.0, 0.1, 0.5]), lens=rng.randrange(1 << 20))
    d = rng.choice([64, 128, 256])
    hk = rng.choice([1, 2, 3, 4, 8])
    if kind == "copy":
        form = rng.choice(["blocks", "tokens"])
        layers = _log_int(rng, 1, 8)
        dtype = rng.choice(["bf16", "fp4"])
        # at most the rows of the largest listed case
        most = 39322 * 4 * 128 // (hk * d * layers)
        entries = _log_int(rng, 1, max(1, min(39322, most) if form == "tokens" else most // block))
        rows = entries * (1 if form == "tokens" else block)
        return dict(kind=kind, form=form, entries=entries, idle=rng.choice([0.0, 0.2]), layers=layers, hk=hk, d=d,
                    block=block, dtype=dtype, tokens=int(rows * rng.uniform(1.0, 3.0)) + block)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    scales = dict(k_scale=rng.choice([1.0, 0.5, 0.3]), v_scale=rng.choice([1.0, 0.25, 0.07]))
    if kind == "append":
        most = max(1, 39322 * 24 * 128 // ((hk * group + 2 * hk) * d))
        return dict(scales, kind=kind, tokens=_log_int(rng, 1, min(39322, most)), hq=hk * group, hk=hk, d=d,
                    rotary=rng.choice([0, 48, d // 4, d // 2, d]), dtype=dtype, block=block,
                    max_pos=_log_int(rng, 40000, 200000))
    form = rng.choice(["decode", "chunk", "prefill", "mixed"])
    case = dict(scales, kind=kind, dtype=dtype, hq=hk * group, hk=hk, d=d, block=block, causal=rng.random() < 0.85,
                window=0, singles=0.0, empty=0.0, lens=rng.randrange(1 << 20))
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


def _offsets(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return off


def _blocks(n, block):
    return -(-n // block)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ 4-bit rows


def _numbers(dtype=torch.float32):
    half = torch.tensor(_NUMBERS, dtype=dtype, device="cuda")
    return torch.cat([half, -half])


def _encode(x):
    """fp32 rows [..., d] -> codes [..., d / 2] and scales [..., d / 16], uint8."""
    x = x.unflatten(-1, (-1, _GROUP))
    scale = (x.abs().amax(-1) / _MOST).clamp(max=448.0).to(torch.float8_e4m3fn)
    scale = torch.where(scale.float() < _LEAST_SCALE, _LEAST_SCALE, scale.float())
    y = x / scale[..., None]
    r = y.abs()
    # halfway between two numbers: the even code
    code = ((r > 0.25).byte() + (r >= 0.75) + (r > 1.25) + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5.0))
    code = (code + 8 * (y < 0)).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes, scales):
    """Values [..., d] in fp32: a number times its scale, which is exact."""
    index = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    values = _numbers()[index].unflatten(-1, (-1, _GROUP))
    return (values * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _parts(pool):
    """Views of a pool's codes [blocks, Hk, bs / 8, 8, d / 2] and scales
    [blocks, Hk, bs / 8, 8, d / 16]."""
    d = pool.shape[-1] * 2 // 9
    return pool[..., :4 * d].unflatten(-1, (8, d // 2)), pool[..., 4 * d:].unflatten(-1, (8, d // 16))


def _pool_values(pool):
    """[blocks, block_size, Hk, d] in fp32, without the pool's factor."""
    return _decode(*_parts(pool)).flatten(2, 3).transpose(1, 2)


def _fill(pool, first, rows):
    """Blocks of a pool from `first` on, from fp32 rows [n, Hk, bs, d]."""
    codes, scales = _parts(pool[first:first + rows.shape[0]])
    c, s = _encode(rows)
    codes.copy_(c.unflatten(2, (-1, 8)))
    scales.copy_(s.unflatten(2, (-1, 8)))


def _new_pool(blocks, bs, hk, d):
    return torch.zeros(blocks, hk, bs // 8, 9 * d // 2, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------ append


def _prepare_append(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, hq, hk, d, bs, rot = (case[x] for x in ("tokens", "hq", "hk", "d", "block", "rotary"))
    dtype = _TYPES[case["dtype"]]
    # one row of queries, keys and values for each token, as a projection leaves
    # it; values are small, some elements of a key head large in every token
    qkv = torch.randn(n, hq + 2 * hk, d, generator=gen, device="cuda")
    qkv[:, hq:hq + hk] *= torch.exp(0.7 * torch.randn(hk, d, generator=gen, device="cuda"))
    qkv[:, hq + hk:] *= 0.3
    qkv = qkv.to(dtype)
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
    pools = [_new_pool(blocks, bs, hk, d) for _ in range(2)]
    for pool in pools:   # what the cache held before
        _fill(pool, 0, torch.randn(blocks, hk, bs, d, generator=gen, device="cuda"))
    return dict(kind="append", rotary=rot, k_scale=case["k_scale"], v_scale=case["v_scale"], dtype=dtype,
                q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], slots=slots, positions=positions,
                cos_sin=table, k_pool=pools[0], v_pool=pools[1],
                q_out=torch.zeros(n, hq, d, dtype=dtype, device="cuda"))


def _plain_append(s):
    half = s["rotary"] // 2

    def rotated(x):
        x = x.float()
        if not half:
            return x
        angle = s["cos_sin"][s["positions"].long()][:, None]
        cos, sin = angle[..., :half], angle[..., half:]
        a, b = x[..., :half], x[..., half:2 * half]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]], -1)

    bs = s["k_pool"].shape[2] * 8
    slots = s["slots"].long()
    block, group, row = slots // bs, slots % bs // 8, slots % 8
    s["q_out"].copy_(rotated(s["q"]))
    k = _stored(s["k_pool"], rotated(s["k"]) / s["k_scale"], block, group, row)
    v = _stored(s["v_pool"], s["v"].float() / s["v_scale"], block, group, row)
    return s["q_out"], (k * s["k_scale"]).to(s["dtype"]), (v * s["v_scale"]).to(s["dtype"])


def _stored(pool, x, block, group, row):
    """Rows x [T, Hk, d] put in their places; the pool's values."""
    for part, new in zip(_parts(pool), _encode(x)):
        part[block, :, group, row] = new
    return _pool_values(pool)


# ------------------------------------------------------------ attention


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
    k_pool, v_pool = _new_pool(blocks, bs, hk, d), _new_pool(blocks, bs, hk, d)
    begins = torch.zeros(blocks, dtype=torch.bool, device="cuda")
    begins[table[torch.tensor([i for i, n in enumerate(used) if n], device="cuda"), 0].long()] = True
    step = max(1, (1 << 26) // (hk * bs * d))
    for at in range(0, blocks, step):
        m = min(step, blocks - at)
        k = torch.randn(m, hk, bs, d, generator=gen, device="cuda")
        k[:, :, 0] = torch.where(begins[at:at + m, None, None], along * 0.8, k[:, :, 0])
        _fill(k_pool, at, k / case["k_scale"])
        _fill(v_pool, at, torch.randn(m, hk, bs, d, generator=gen, device="cuda"))
    tokens = sum(new)
    q = torch.randn(tokens, hk, hq // hk, d, generator=gen, device="cuda", dtype=torch.float32) * 1.5
    q = (q + 0.5 * along[:, None]).reshape(tokens, hq, d)
    s = dict(kind="attention", causal=case["causal"], window=case["window"], tokens=tokens, max_new=max(new),
             max_kv=max(kv), k_scale=case["k_scale"], v_scale=case["v_scale"], q=q.to(dtype), k_pool=k_pool,
             v_pool=v_pool, table=table, kv_len=_i32(kv), q_off=_i32(_offsets(new)),
             out=torch.zeros(tokens, hq, d, dtype=dtype, device="cuda"),
             lse=torch.zeros(tokens, hq, dtype=torch.float32, device="cuda"), ws=None)
    if own:
        import speculative_prefill_token_gb300 as sp
        # a server knows how many tokens a request adds at most, and how many its chunks see
        s["ws"] = sp.make_attention_fp4_workspace(s["q"], len(new), s["k_pool"], max_new=s["max_new"],
                                                  kv_tokens=sum(kv))
    return s


def _plain_attention(s):
    q, table = s["q"], s["table"]
    tokens, hq, d = q.shape
    hk, bs = s["k_pool"].shape[1], s["k_pool"].shape[2] * 8
    g = hq // hk
    off, kv = s["q_off"].long(), s["kv_len"].long()
    new = off[1:] - off[:-1]
    batch = kv.numel()
    # the cached rows of every request, [B, Hk, keys, d]; zeros behind its end
    j = torch.arange(s["max_kv"], device="cuda")
    there = j < kv[:, None]
    pages = table[:, :_blocks(s["max_kv"], bs)].long()

    def cached(pool):
        rows = _decode(*_parts(pool[pages].transpose(1, 2)))   # [B, Hk, pages, bs / 8, 8, d]
        return rows.flatten(2, 4)[:, :, :s["max_kv"]].masked_fill(~there[:, None, :, None], 0.0)

    keys, values = cached(s["k_pool"]), cached(s["v_pool"])
    # the new tokens of every request, [B, Hk, G * new, d]
    i = torch.arange(s["max_new"], device="cuda")
    index = (off[:-1, None] + i).clamp(max=tokens - 1)
    qs = q[index].float().view(batch, -1, hk, g, d).permute(0, 2, 3, 1, 4).reshape(batch, hk, -1, d)
    scores = torch.matmul(qs, keys.transpose(2, 3)).view(batch, hk, g, -1, s["max_kv"]) * (s["k_scale"] * d ** -0.5)
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
    o = torch.where(total > 0, o / total, 0.0) * s["v_scale"]
    lse = (torch.log(total) + top)[..., 0]
    t = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(off[1:], t, right=True).clamp(max=batch - 1)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4)[b, t - off[b]].reshape(tokens, hq, d))
    s["lse"].copy_(lse.permute(0, 3, 1, 2)[b, t - off[b]].reshape(tokens, hq))
    return s["out"], s["lse"]


# ------------------------------------------------------------ copies


def _prepare_copy(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, hk, d, bs = (case[x] for x in ("entries", "hk", "d", "block"))
    tokens = case["form"] == "tokens"
    held = _blocks(max(case["tokens"], n * (1 if tokens else bs)), bs)
    fresh = _blocks(n, bs) if tokens else n
    blocks = held + fresh + 3
    ids = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    table, src_off = None, None
    if tokens:
        # kept tokens of a cached prompt, in two requests, to blocks of their own
        cut = n // 3
        first = (held + 1) // 2
        table = torch.stack([ids[:first], ids[held - first:held]]).contiguous()
        span = first * bs
        src = torch.cat([torch.randperm(span, generator=gen, device="cuda")[:m].sort().values
                         for m in (min(cut, span), min(n - cut, span))]).to(torch.int32)
        n = src.numel()
        src_off = _i32([0, min(cut, span), n])
        t = torch.arange(n, device="cuda")
        dst = ids[held:held + fresh].long()[t // bs] * bs + t % bs
        dst = dst.to(torch.int32)
    else:
        src, dst = ids[:n].clone(), ids[held:held + n].clone()
    idle = torch.rand(n, generator=gen, device="cuda") < case["idle"]
    dst[idle] = -1
    shape = (blocks, hk, bs // 8, 9 * d // 2) if case["dtype"] == "fp4" else (blocks, bs, hk, d)
    pools = []
    for _ in range(2 * case["layers"]):
        if case["dtype"] == "fp4":   # (a copy moves bytes, whatever they stand for: they come back as they are)
            pool = torch.randint(0, 127, shape, generator=gen, device="cuda", dtype=torch.uint8)
        else:
            pool = torch.randn(shape, generator=gen, device="cuda").to(_TYPES[case["dtype"]])
        pools.append(pool)
    return dict(kind="copy", fp4=case["dtype"] == "fp4", block=bs, rows=1 if tokens else bs, pools=pools, src=src,
                dst=dst, table=table, src_off=src_off)


def _plain_copy(s):
    src, dst, bs = s["src"].long(), s["dst"].long(), s["block"]
    if s["table"] is not None:
        i = torch.arange(src.numel(), device="cuda")
        b = torch.searchsorted(s["src_off"][1:].long(), i, right=True)
        src = s["table"][b, src // bs].long() * bs + src % bs
    # an entry that copies nothing writes a row to itself
    dst = torch.where(dst < 0, src, dst)
    for pool in s["pools"]:
        if s["rows"] > 1:
            pool[dst] = pool[src]
        elif s["fp4"]:
            for part in _parts(pool):
                part[dst // bs, :, dst % bs // 8, dst % 8] = part[src // bs, :, src % bs // 8, src % 8]
        else:
            rows = pool.flatten(0, 1)
            rows[dst] = rows[src]
    return s["pools"]


# ------------------------------------------------------------ pages


def _prepare_pages(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(case["lens"])
    bs, parents, forks = case["block"], case["parents"], case["forks"]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(parents)]
    held = [_blocks(c, bs) for c in ctx]
    spare = parents * forks + 5
    pool_blocks = sum(held) + spare
    ids = torch.randperm(pool_blocks, generator=gen, device="cuda").to(torch.int32)
    width = max(max(held), 1) + 2
    rows = parents * (forks + 1)
    col = torch.arange(width, device="cuda")
    first = torch.tensor(_offsets(held)[:-1], device="cuda")
    table = torch.full((rows, width), -7, dtype=torch.int32, device="cuda")   # stale where nothing is held
    # requests and free rows lie in any order
    order = torch.randperm(rows, generator=gen, device="cuda")
    at = order[:parents]
    table[at] = torch.where(col < torch.tensor(held, device="cuda")[:, None],
                            ids[(first[:, None] + col).clamp(max=pool_blocks - 1)], -7)
    ctx_len = torch.zeros(rows, dtype=torch.int32, device="cuda")
    ctx_len[at] = _i32(ctx)
    src = at.repeat_interleave(forks).to(torch.int32)
    dst = order[parents:].to(torch.int32)
    src[torch.rand(src.numel(), generator=gen, device="cuda") < case["idle"]] = -1
    free = torch.zeros(pool_blocks, dtype=torch.int32, device="cuda")
    free[:spare] = ids[sum(held):]
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    # the first block of a request may be shared with requests elsewhere
    shared = i32(pool_blocks)
    some = at[torch.tensor([i for i, n in enumerate(held) if n], device="cuda", dtype=torch.long)]
    shared[table[some, 0].long()] = torch.randint(0, 3, (some.numel(),), generator=gen, device="cuda",
                                                  dtype=torch.int32)
    return dict(kind="pages", block=bs, src=src, dst=dst, ctx_len=ctx_len, table=table, shared=shared, free=free,
                n_free=_i32([spare]), kv_len=i32(rows), copy_src=i32(src.numel()), copy_dst=i32(src.numel()),
                n_left=i32(1), len_after=i32(rows), n_after=i32(1))


def _plain_pages(s):
    bs, table, shared = s["block"], s["table"], s["shared"]
    n_free = s["n_free"].long()
    live = s["src"] >= 0
    src, dst = s["src"].clamp(min=0).long(), s["dst"].long()
    length = torch.where(live, s["ctx_len"][src], 0).long()
    full, begun = length // bs, length % bs > 0
    before = torch.cumsum(begun, 0) - begun.long()
    fresh = s["free"][(n_free - 1 - before).clamp(min=0)]
    col = torch.arange(table.shape[1], device="cuda")
    share = live[:, None] & (col < full[:, None])
    shared.scatter_add_(0, torch.where(share, table[src], 0).long().flatten(), share.flatten().int())
    s["copy_src"].copy_(torch.where(begun, table[src, full.clamp(max=table.shape[1] - 1)], -1))
    s["copy_dst"].copy_(torch.where(begun, fresh, -1))
    new = begun[:, None] & (col == full[:, None])
    table[dst] = torch.where(share, table[src], torch.where(new, fresh[:, None], table[dst]))
    s["kv_len"].copy_(s["ctx_len"])
    s["kv_len"][dst] = torch.where(live, length.int(), s["ctx_len"][dst])
    s["n_left"].copy_(n_free - begun.sum())
    forked = table.clone(), shared.clone()
    # the forks end: back to the lengths before them
    held, keep = (s["kv_len"].long() + bs - 1) // bs, (s["ctx_len"].long() + bs - 1) // bs
    drop = (col >= keep[:, None]) & (col < held[:, None])
    drops = torch.zeros_like(shared).scatter_add_(0, torch.where(drop, table, 0).long().flatten(), drop.flatten().int())
    freed = drops > shared
    shared.copy_(torch.where(freed, 0, shared - drops))
    # blocks that nobody holds any more, in the order of their ids
    place = torch.where(freed, s["n_left"].long() + torch.cumsum(freed, 0) - 1, s["free"].numel())
    longer = torch.cat([s["free"], s["free"][:1]])
    longer[place] = torch.arange(shared.numel(), dtype=torch.int32, device="cuda")
    s["free"].copy_(longer[:-1])
    s["n_after"].copy_(s["n_left"] + freed.sum())
    s["len_after"].copy_(s["ctx_len"])
    return (*forked, s["copy_src"], s["copy_dst"], s["kv_len"], s["n_left"], shared, s["free"], s["len_after"],
            s["n_after"])


# ------------------------------------------------------------ the cases


def prepare(case, seed):
    return {"append": _prepare_append, "attention": _prepare_attention, "copy": _prepare_copy,
            "pages": _prepare_pages}[case["kind"]](case, seed)


def _own(s):
    import speculative_prefill_token_gb300 as sp
    if s["kind"] == "append":
        sp.append_kv_fp4(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], q=s["q"], q_out=s["q_out"],
                         positions=s["positions"] if s["rotary"] else None, cos_sin=s["cos_sin"],
                         k_scale=s["k_scale"], v_scale=s["v_scale"])
        return (s["q_out"], sp.unpack_fp4(s["k_pool"], s["dtype"], scale=s["k_scale"]),
                sp.unpack_fp4(s["v_pool"], s["dtype"], scale=s["v_scale"]))
    if s["kind"] == "attention":
        sp.paged_attention_fp4(s["q"], s["q_off"], s["kv_len"], s["table"], s["k_pool"], s["v_pool"],
                               causal=s["causal"], window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                               out=s["out"], lse=s["lse"], max_new=s["max_new"], ws=s["ws"])
        return s["out"], s["lse"]
    if s["kind"] == "copy":
        sp.copy_kv(s["pools"], s["src"], s["dst"], rows=s["rows"], block_table=s["table"], src_off=s["src_off"])
        return s["pools"]
    sp.fork_blocks(s["src"], s["dst"], s["ctx_len"], s["table"], s["shared"], s["free"], s["n_free"], s["block"],
                   kv_len=s["kv_len"], copy_src=s["copy_src"], copy_dst=s["copy_dst"], n_left=s["n_left"])
    forked = s["table"].clone(), s["shared"].clone()
    sp.free_blocks(s["kv_len"], s["ctx_len"], s["table"], s["shared"], s["free"], s["n_left"], s["block"],
                   kv_len=s["len_after"], n_left=s["n_after"])
    return (*forked, s["copy_src"], s["copy_dst"], s["kv_len"], s["n_left"], s["shared"], s["free"], s["len_after"],
            s["n_after"])


def run(s):
    if own:
        return _own(s)
    return {"append": _plain_append, "attention": _plain_attention, "copy": _plain_copy,
            "pages": _plain_pages}[s["kind"]](s)


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
        n, hq, hk, d, bs = (case[x] for x in ("tokens", "hq", "hk", "d", "block"))
        rows = (_blocks(n, bs) + 3) * bs
        # queries, keys and values in, queries and 4-bit rows out; the pools' values out again
        return {"bytes": 2 * n * (2 * hq + 2 * hk) * d + n * (8 + 4 * case["rotary"]) + 9 * n * hk * d // 8
                + 9 * rows * hk * d // 8 + 4 * rows * hk * d, "flops": 3 * n * (hq + hk) * case["rotary"]}
    if case["kind"] == "copy":
        hk, d = case["hk"], case["d"]
        n = int(case["entries"] * (1 - case["idle"]))
        rows = n * (1 if case["form"] == "tokens" else case["block"])
        size = 9 * d // 16 if case["dtype"] == "fp4" else 2 * d
        return {"bytes": 4 * case["layers"] * rows * hk * size + 8 * case["entries"], "flops": 0}
    if case["kind"] == "pages":
        rng = random.Random(case["lens"])
        ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["parents"])]
        held = sum(_blocks(c, case["block"]) for c in ctx)
        blocks = held + case["parents"] * case["forks"] + 5
        forks = case["forks"] * (1 - case["idle"])
        rows = case["parents"] * (case["forks"] + 1)
        # the parents' blocks read and the forks' written and read, a count of each read and written
        # twice, and the copies of tables and counts that are handed back
        width = max(_blocks(c, case["block"]) for c in ctx) + 2
        return {"bytes": int(4 * held * (1 + 2 * forks + 4)) + 8 * (rows * width + blocks) + 20 * rows, "flops": 0}
    ctx, new = _lengths(case)
    pairs, keys = _pairs(case, ctx, new)
    hq, hk, d = case["hq"], case["hk"], case["d"]
    table = sum(_blocks(c + n, case["block"]) for c, n in zip(ctx, new))
    return {"bytes": 2 * 9 * keys * hk * d // 16 + 2 * 2 * sum(new) * hq * d + 4 * sum(new) * hq + 4 * table
            + 8 * len(ctx), "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------ in 64 bits


def _value64(pool):
    """A pool's values in 64 bits, [blocks, Hk, bs, d], from its bits."""
    blocks, hk, groups, width = pool.shape
    d = width * 2 // 9
    code = pool[..., :4 * d].reshape(blocks, hk, groups * 8, d // 2)
    both = torch.stack([code % 16, code // 16], -1).reshape(blocks, hk, groups * 8, d).int()
    e, m = both // 2 % 4, (both % 2).double()
    size = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
    byte = pool[..., 4 * d:].reshape(blocks, hk, groups * 8, d // 16).int()
    e, m = byte // 8 % 16, (byte % 8).double()
    scale = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2(e.double() - 7))
    return torch.where(both > 7, -size, size) * scale.repeat_interleave(16, -1)


def _rounded64(x):
    """Rows [..., d] in 64 bits as 4 bits hold them."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    want = g.abs().amax(-1, keepdim=True) / 6
    # e4m3: steps of 2^(exponent - 3), of 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3)
    scale = (torch.round(want / step) * step).clamp(2.0 ** -9, 448.0)
    r = g / scale
    # e2m1: steps of a half below 2, of 1 below 4, of 2 above
    a = r.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.sign(r) * (torch.round(a / step) * step).clamp(max=6.0) * scale).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "append":
        r = case["rotary"] // 2
        rows = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            if r:
                z = torch.complex(y[..., :r], y[..., r:2 * r])
                turn = s["cos_sin"].double()[s["positions"].long()]
                z = z * torch.complex(turn[:, :r], turn[:, r:])[:, None]
                y[..., :r], y[..., r:2 * r] = z.real, z.imag
            rows.append(y)
        pools = []
        for pool, x, f in ((s["k_pool"], rows[1], case["k_scale"]), (s["v_pool"], s["v"].double(), case["v_scale"])):
            whole = _value64(pool).transpose(1, 2).reshape(-1, case["hk"], case["d"])
            whole[s["slots"].long()] = _rounded64(x / f)
            pools.append((whole * f).reshape(-1, case["block"], case["hk"], case["d"]))
        return rows[0], pools[0], pools[1]
    if case["kind"] == "copy":
        src, dst = s["src"].tolist(), s["dst"].tolist()
        if s["table"] is not None:
            cut, table, bs = s["src_off"].tolist()[1], s["table"].tolist(), case["block"]
            src = [table[int(i >= cut)][t // bs] * bs + t % bs for i, t in enumerate(src)]
        pairs = [(a, b) for a, b in zip(src, dst) if b >= 0]
        take, put = (torch.tensor(x, device="cuda") for x in zip(*pairs)) if pairs else (None, None)
        out = []
        for pool in s["pools"]:
            old, new = pool, pool.clone()
            if case["form"] == "blocks":
                if pairs:
                    new[put] = old[take]
            elif case["dtype"] == "fp4":
                d, bs = case["d"], case["block"]
                for lo, n in ((0, d // 2), (4 * d, d // 16)):
                    byte = torch.arange(n, device="cuda")
                    new[(put // bs)[:, None], :, (put % bs // 8)[:, None], lo + (put % 8)[:, None] * n + byte] = \
                        old[(take // bs)[:, None], :, (take % bs // 8)[:, None], lo + (take % 8)[:, None] * n + byte]
            else:
                new.view(-1, case["hk"], case["d"])[put] = old.view(-1, case["hk"], case["d"])[take]
            out.append(new.double() if case["dtype"] != "fp4" else new)
        return out
    if case["kind"] == "pages":
        return None   # whole numbers
    ctx, new = _lengths(case)
    hq, hk, d, bs = (case[x] for x in ("hq", "hk", "d", "block"))
    g = hq // hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    first = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        pages = s["table"][b, :_blocks(c + n, bs)].long()
        for h in range(hk if n else 0):
            k = _value64(s["k_pool"][pages, h:h + 1]).reshape(-1, d)[:c + n] * case["k_scale"]
            v = _value64(s["v_pool"][pages, h:h + 1]).reshape(-1, d)[:c + n] * case["v_scale"]
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
