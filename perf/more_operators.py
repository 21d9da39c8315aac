"""Cases of a request's way into a paged KV cache and out of it again.

Four operators, each in a plain form (elementary torch operations in 32 bits, in 64 where a value is
cut to 8 or 4 bits and may lie next to the border of two) and as a user calls it from
``varlen_top_select_amd``:

  write    write_cache       head norms and rotary positions of q and k, K and V written to their slots
                             in 16 bits or microscaled in 8 or 4, and read back with read_cache
  read     read_cache        cached rows of listed slots, as 16-bit rows
  attend   tree_attention    drafted tokens over a microscaled cache
  prompt   prompt_attention  packed prompts, causal, grouped heads

A microscaled row holds one power of two per 32 elements (E8M0, a byte) and elements of 8 bits (E4M3) or
4 (E2M1, the first of two in the low half of a byte).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
POSITIONS = 32768  # rows of the rotary table


def listed():
    return [
        # one token of one request enters a 4-bit cache: all latency
        dict(name="write_token", op="write", tokens=1, heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, norm=True, keep_k=False, page=64, bits=4, heads_first=False, pad=False, dtype="bf16"),
        # a prompt's 16384 tokens; the rotated keys are returned too, for the prompt's own attention
        dict(name="write_prompt", op="write", tokens=16384, heads=64, kv_heads=8, dim=128, rot=128,
             interleaved=False, norm=True, keep_k=True, page=64, bits=4, heads_first=False, pad=False, dtype="bf16"),
        # odd everything: half the head rotated in neighbouring pairs, pages of 24, padding tokens, 8 bits
        dict(name="write_odd", op="write", tokens=1001, heads=14, kv_heads=2, dim=64, rot=32,
             interleaved=True, norm=False, keep_k=False, page=24, bits=8, heads_first=False, pad=True, dtype="fp16"),
        # a long context read back in front of the next chunk of its prompt
        dict(name="read_context", op="read", slots=65536, kv_heads=8, dim=128, page=64, bits=4,
             heads_first=False, dtype="bf16"),
        # a few hundred selected entries
        dict(name="read_few", op="read", slots=300, kv_heads=2, dim=64, page=24, bits=8,
             heads_first=False, dtype="fp16"),
        # one request, one token over a 4-bit cache: the smallest decode step
        dict(name="attend_single", op="attend", batch=1, draft=1, heads=32, kv_heads=8, dim=128,
             page=64, longest=4096, tree=False, top_k=0, bits=4, heads_first=False, dtype="bf16"),
        # a served batch with one drafted token after the real one, ragged lengths
        dict(name="attend_chain", op="attend", batch=64, draft=2, heads=64, kv_heads=8, dim=128,
             page=64, longest=16384, tree=False, top_k=0, bits=4, heads_first=False, dtype="bf16"),
        # a tree of 16 drafted tokens over long contexts, a cache laid out heads first
        dict(name="attend_tree_long", op="attend", batch=8, draft=16, heads=64, kv_heads=8, dim=128,
             page=64, longest=65536, tree=True, top_k=0, bits=4, heads_first=True, dtype="bf16"),
        # each drafted row attends 2048 selected slots of an 8-bit cache, and its ancestors
        dict(name="attend_slots", op="attend", batch=64, draft=2, heads=64, kv_heads=4, dim=128,
             page=64, longest=65536, tree=True, top_k=2048, bits=8, heads_first=False, dtype="bf16"),
        # one long prompt
        dict(name="prompt_long", op="prompt", batch=1, longest=16384, shortest=16384, context=0,
             heads=32, kv_heads=8, dim=128, causal=True, dtype="bf16"),
        # many prompts packed, from one token up, odd heads, head size 64
        dict(name="prompt_packed", op="prompt", batch=61, longest=2500, shortest=1, context=0,
             heads=14, kv_heads=2, dim=64, causal=True, dtype="fp16"),
        # the next 512 tokens of eight prompts behind what is cached of them
        dict(name="prompt_chunk", op="prompt", batch=8, longest=512, shortest=512, context=16384,
             heads=64, kv_heads=8, dim=128, causal=True, dtype="bf16"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["write", "read", "attend", "attend", "prompt", "prompt"])
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 3, 4, 7, 8])
    page = rng.choice([1, 16, 24, 64, 64, 128])
    bits = rng.choice([4, 4, 8])
    heads_first = rng.random() < 0.3
    if op == "write":
        rot = rng.choice([0, 32, dim // 2, dim, dim])
        return dict(op=op, tokens=log(1, 16384), heads=group * kv_heads, kv_heads=kv_heads, dim=dim,
                    rot=rot, interleaved=rng.random() < 0.3, norm=rng.random() < 0.6,
                    keep_k=rng.random() < 0.5, page=page, bits=rng.choice([4, 8, 16]),
                    heads_first=heads_first, pad=rng.random() < 0.3, dtype=dtype)
    if op == "read":
        return dict(op=op, slots=log(1, 65536), kv_heads=kv_heads, dim=dim, page=page,
                    bits=rng.choice([4, 8, 16]), heads_first=heads_first, dtype=dtype)
    if op == "prompt":
        batch = log(1, 64)
        longest = min(log(16, 8192), 65536 // batch)
        context = rng.choice([0, 0, log(100, 16384)])
        context = min(context, 131072 // batch)
        case = dict(op=op, batch=batch, longest=longest, shortest=rng.randint(1, longest),
                    context=context, heads=group * kv_heads, kv_heads=kv_heads, dim=dim,
                    causal=rng.random() < 0.8, dtype=dtype)
        while work(case)["flops"] > 2e12:
            case["context"] //= 2
            case["longest"] = case["longest"] * 3 // 4
            case["shortest"] = min(case["shortest"], case["longest"])
        return case
    batch = log(1, 64)
    longest = min(log(100, 65536), 16384 * 64 // batch)
    draft = rng.randint(1, 16 if batch <= 8 else 4)
    while draft * group * kv_heads > 1024 // (1 if batch <= 8 else 8):
        group = max(1, group // 2)
        draft = max(1, draft - 1)
    top_k = log(64, 2048) if rng.random() < 0.35 else 0
    return dict(op=op, batch=batch, draft=draft, heads=group * kv_heads, kv_heads=kv_heads, dim=dim,
                page=page, longest=longest, tree=rng.random() < 0.6, top_k=top_k, bits=bits,
                heads_first=heads_first, dtype=dtype)


# ---------------------------------------------------------------------------- microscaled rows

def power(e, dtype):
    """2^e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64).to(dtype)


def scales_of(top, bits):
    """The exponent of a block whose largest magnitude is `top`: the least with which that rounds to a
    number of the format; and whether the block is finite."""
    fine = torch.isfinite(top)
    part, e = torch.frexp(torch.where(fine, top, 0.0))  # top = part * 2^e, part in [0.5, 1)
    e = e - 3 + (part >= 0.875).int() if bits == 4 else e - 9 + (part > 0.90625).int()
    return torch.where(part == 0, -127, e).clamp(-127, 127), fine


def rounded(x, bits):
    """x rounded to the nearest number of the format, ties to the even one."""
    _, e = torch.frexp(x)
    step = (e - 2).clamp(min=-1) if bits == 4 else (e - 4).clamp(min=-9)
    return torch.round(x * power(-step, x.dtype)) * power(step, x.dtype)


def quantised(x, bits):
    """(elements, exponents, finite) of rows x [..., D]; elements as numbers of the format."""
    blocks = x.unflatten(-1, (-1, 32))
    e, fine = scales_of(blocks.abs().amax(-1), bits)
    scaled = torch.where(fine[..., None], blocks, 0.0) * power(-e[..., None], x.dtype)
    return rounded(scaled, bits), e, fine


def codes(elements, bits):
    """The bytes of elements [..., blocks, 32]: a row's blocks one after the other."""
    if bits == 8:
        return elements.float().to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    size = elements.abs().float()
    code = (2 * size.clamp(max=2) + (size.clamp(2, 4) - 2) + (size.clamp(4, 6) - 4) / 2).to(torch.uint8)
    code = code | (elements < 0).to(torch.uint8) << 3
    code = code.flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4


def values(data, scale, bits):
    """fp32 values of bytes [..., row] with scales [..., D / 32]."""
    if bits == 8:
        x = data.view(torch.float8_e4m3fn).float()
    else:
        half = torch.stack([data & 15, data >> 4], -1).flatten(-2)
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=data.device)
        x = table[(half & 7).long()] * (1 - 2 * (half >> 3).float())
    x = x.unflatten(-1, (-1, 32)) * power(scale.int()[..., None] - 127, x.dtype)
    return torch.where((scale == 255)[..., None], math.nan, x).flatten(-2)


def row_bytes(case):
    return case["dim"] * case["bits"] // 8


# ---------------------------------------------------------------------------- inputs

def cache_memory(case, pool, width, dtype, gen, fill):
    """A cache tensor [pages, page, heads, width]; laid out heads first it is a permuted view."""
    dev = torch.device("cuda")
    if case["heads_first"]:
        t = torch.empty(pool, case["kv_heads"], case["page"], width, dtype=dtype, device=dev).transpose(1, 2)
    else:
        t = torch.empty(pool, case["page"], case["kv_heads"], width, dtype=dtype, device=dev)
    return t.fill_(fill)


def filled_cache(case, pool, gen):
    """(cache, scales or None) with normally distributed entries."""
    dev = torch.device("cuda")
    bits, dim = case["bits"], case["dim"]
    shape = (pool, case["page"], case["kv_heads"])
    if bits == 16:
        data = cache_memory(case, pool, dim, DTYPES[case["dtype"]], gen, 0)
        data.copy_(torch.randn(*shape, dim, generator=gen, device=dev))
        return data, None
    data = cache_memory(case, pool, row_bytes(case), torch.uint8, gen, 0)
    scales = cache_memory(case, pool, dim // 32, torch.uint8, gen, 0)
    each = max(1, (1 << 27) // (case["page"] * case["kv_heads"] * dim))
    for p in range(0, pool, each):  # (the 32-bit values of all pages would be several times the cache)
        x = torch.randn(min(each, pool - p), *shape[1:], dim, generator=gen, device=dev)
        elements, e, _ = quantised(x, bits)
        data[p:p + each] = codes(elements, bits)
        scales[p:p + each] = (e + 127).to(torch.uint8)
    return data, scales


def lengths(case):
    """The batch's lengths, spread over their range; the seed only changes their order."""
    n, hi = case["batch"], case["longest"]
    lo = max(case["draft"], hi // 3) if case["op"] == "attend" else case["shortest"]
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def paged(case, gen, dev):
    """Lengths in the seed's order and a page table whose pages lie in any order of the pool."""
    n, page = case["batch"], case["page"]
    lens = torch.tensor(lengths(case), device=dev)
    lens = lens[torch.randperm(n, generator=gen, device=dev)]
    width = -(-case["longest"] // page)
    used = (lens + page - 1) // page
    pool = int(sum(-(-x // page) for x in lengths(case))) + 3
    order = torch.randperm(pool, generator=gen, device=dev)
    start = torch.cumsum(used, 0) - used
    entry = torch.arange(width, device=dev)
    at = start[:, None] + entry[None]
    table = torch.where(entry[None] < used[:, None], order[at.clamp(max=pool - 1)], -1)
    return lens.to(torch.int32), table.to(torch.int32).contiguous(), pool


def random_tree_bits(n, draft, gen, dev):
    """Each node's ancestors and itself as bits of an int64; a node's parent is an earlier one, or none."""
    node = torch.arange(draft, device=dev)
    low = torch.clamp((node - 1) // 3, min=0)
    pick = torch.rand(n, draft, generator=gen, device=dev)
    parent = (low + (pick * (node - low)).long()).clamp(max=draft) - 1
    parent = torch.minimum(parent, node[None] - 1)
    bits = torch.zeros(n, draft, dtype=torch.int64, device=dev)
    for t in range(draft):
        up = bits.gather(1, parent[:, t].clamp(min=0)[:, None])[:, 0]
        bits[:, t] = torch.where(parent[:, t] >= 0, up, 0) | (1 << t)
    return bits


def rotary(rot, dev):
    """[POSITIONS, rot]: cosines, then sines."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    angle = torch.arange(POSITIONS, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat([torch.cos(angle), torch.sin(angle)], 1).float().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    kv, dim = case["kv_heads"], case["dim"]
    s = {"case": case}

    def normal(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=gen, device=dev)).to(dtype)

    if case["op"] == "write":
        n, heads, page = case["tokens"], case["heads"], case["page"]
        # views of one projection's output, as a model has them
        qkv = normal(n, heads + 2 * kv, dim, scale=2.0)
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        first = int(torch.randint(0, POSITIONS - n + 1, (1,), generator=gen, device=dev))
        s["positions"] = s["rotary"] = None
        if case["rot"]:
            s["positions"] = torch.arange(first, first + n, device=dev, dtype=torch.int32)
            s["rotary"] = rotary(case["rot"], dev)
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = (1 + 0.3 * torch.randn(dim, generator=gen, device=dev)).to(dtype)
            s["k_norm"] = (1 + 0.3 * torch.randn(dim, generator=gen, device=dev)).to(dtype)
        pool = -(-n // page) + 3
        # the request's pages lie anywhere
        order = torch.randperm(pool, generator=gen, device=dev)
        pos = torch.arange(n, device=dev)
        slots = order[pos // page] * page + pos % page
        if case["pad"]:
            slots = torch.where(torch.rand(n, generator=gen, device=dev) < 0.1, -1, slots)
        s["slots"] = slots.to(torch.int32)
        width = dim if case["bits"] == 16 else row_bytes(case)
        kind = dtype if case["bits"] == 16 else torch.uint8
        s["k_cache"], s["v_cache"] = (cache_memory(case, pool, width, kind, gen, 0) for _ in "kv")
        s["k_scales"] = s["v_scales"] = None
        if case["bits"] != 16:
            s["k_scales"], s["v_scales"] = (
                cache_memory(case, pool, dim // 32, torch.uint8, gen, 0) for _ in "kv")
        return s
    if case["op"] == "read":
        page = case["page"]
        pool = -(-case["slots"] // page) + 3
        s["k_cache"], s["k_scales"] = filled_cache(case, pool, gen)
        s["v_cache"], s["v_scales"] = filled_cache(case, pool, gen)
        order = torch.randperm(pool, generator=gen, device=dev)
        pos = torch.arange(case["slots"], device=dev)
        s["slots"] = (order[pos // page] * page + pos % page).to(torch.int32)
        return s
    if case["op"] == "prompt":
        lens = torch.tensor(lengths(case), device=dev)
        lens = lens[torch.randperm(case["batch"], generator=gen, device=dev)]
        before = torch.tensor(contexts(case), device=dev)
        zero = torch.zeros(1, dtype=torch.long, device=dev)
        s["cu_q"] = torch.cat([zero, torch.cumsum(lens, 0)]).to(torch.int32)
        s["cu_k"] = torch.cat([zero, torch.cumsum(lens + before, 0)]).to(torch.int32)
        total_q = sum(lengths(case))
        total_k = total_q + sum(contexts(case))
        s["q"] = normal(total_q, case["heads"], dim, scale=1.5)
        s["k"], s["v"] = normal(total_k, kv, dim), normal(total_k, kv, dim)
        s["scale"] = 1.0 / math.sqrt(dim)
        return s

    n, draft, heads, page = case["batch"], case["draft"], case["heads"], case["page"]
    s["lens"], s["table"], pool = paged(case, gen, dev)
    s["k_cache"], s["k_scales"] = filled_cache(case, pool, gen)
    s["v_cache"], s["v_scales"] = filled_cache(case, pool, gen)
    s["q"] = normal(n, draft, heads, dim, scale=1.5)
    s["scale"] = 1.0 / math.sqrt(dim)
    s["mask"] = random_tree_bits(n, draft, gen, dev) if case["tree"] else None
    s["slots"] = None
    if case["top_k"]:
        k = min(case["top_k"], case["longest"])
        score = torch.rand(n * draft, case["longest"], generator=gen, device=dev)
        col = torch.arange(case["longest"], device=dev)
        prefix = (s["lens"].long() - draft).repeat_interleave(draft)
        score = torch.where(col[None] < prefix[:, None], score, -1.0)
        best, at = torch.topk(score, k, dim=-1, sorted=False)
        entry = s["table"].long().repeat_interleave(draft, 0).gather(1, at // page)
        slot = torch.where(best >= 0, entry * page + at % page, -1)
        # unused slots come last, as the selection writes them
        order = torch.argsort((slot < 0).int(), dim=-1, stable=True)
        s["slots"] = slot.gather(1, order).to(torch.int32).view(n, draft, k).contiguous()
    return s


def contexts(case):
    """The number of cached entries in front of each prompt, from half of `context` to all of it."""
    n = case["batch"]
    return [int((0.5 + 0.5 * i / (n - 1) if n > 1 else 0.5) * case["context"]) for i in range(n)]


# ---------------------------------------------------------------------------- plain forms

def turned(x, table, positions, interleaved):
    """Rows x [T, H, D] turned by their positions' angles."""
    rot = table.shape[1]
    cos, sin = table[positions.long()].to(x.dtype)[:, None].chunk(2, -1)
    part = x[..., :rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else part.chunk(2, -1)
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y, x[..., rot:]], -1)


def plain_write(s):
    c = s["case"]
    bits, dtype = c["bits"], s["q"].dtype

    def normed(x, w):
        if w is None:
            return x
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.to(x.dtype)

    def done(x, w):
        x = normed(x, w)
        return x if s["rotary"] is None else turned(x, s["rotary"], s["positions"], c["interleaved"])

    def cached(x):
        if bits == 16:
            return x.to(dtype)
        elements, e, _ = quantised(x, bits)
        return (elements * power(e[..., None], x.dtype)).flatten(-2).to(dtype)

    q = done(s["q"].float(), s["q_norm"]).to(dtype)
    k = done(s["k"].double(), s["k_norm"])
    kept = (s["slots"] >= 0)[:, None, None]
    out = {"q": q, "k_cached": torch.where(kept, cached(k), 0.0),
           "v_cached": torch.where(kept, cached(s["v"].double()), 0.0)}
    if c["keep_k"]:
        out["k"] = k.to(dtype)
    return out


def rows_of(s, which, slot):
    """fp32 rows [..., heads, D] of the slots of one of the two caches."""
    page, bits = s["case"]["page"], s["case"]["bits"]
    x = s[which + "_cache"][slot // page, slot % page]
    return x.float() if bits == 16 else values(x, s[which + "_scales"][slot // page, slot % page], bits)


def plain_read(s):
    dtype, slot = DTYPES[s["case"]["dtype"]], s["slots"].long()
    return {"k": rows_of(s, "k", slot).to(dtype), "v": rows_of(s, "v", slot).to(dtype)}


def visible_drafts(mask, n, draft, dev):
    """[n, t, i]: row t sees drafted token i."""
    i = torch.arange(draft, device=dev)
    if mask is None:
        return (i[None] <= i[:, None])[None].expand(n, -1, -1)
    return ((mask[:, :, None] >> i) & 1).bool()


def dense_plan(s):
    """Slot and visibility of every position of each request: [n, S], [n, t, S]."""
    dev, page = s["table"].device, s["case"]["page"]
    n, draft = s["case"]["batch"], s["case"]["draft"]
    lens = s["lens"].long()
    pos = torch.arange(s["case"]["longest"], device=dev)
    entry = s["table"].long()[:, pos // page]
    slot = entry.clamp(min=0) * page + pos % page
    i = pos[None] - (lens - draft)[:, None]
    tree = visible_drafts(s["mask"], n, draft, dev)
    tree = tree.gather(2, i.clamp(0, draft - 1)[:, None].expand(-1, draft, -1))
    vis = torch.where((i < 0)[:, None], True, tree & (i < draft)[:, None])
    return slot, vis & (entry >= 0)[:, None]


def slots_plan(s):
    """The same for slot lists: every row is a request of its own with one row of queries."""
    dev, page = s["table"].device, s["case"]["page"]
    n, draft = s["case"]["batch"], s["case"]["draft"]
    slot = s["slots"].long().view(n * draft, -1)
    vis = slot >= 0
    if s["mask"] is not None:
        pos = (s["lens"].long() - draft)[:, None] + torch.arange(draft, device=dev)
        entry = s["table"].long().gather(1, pos.clamp(min=0) // page)
        own_slot = (entry.clamp(min=0) * page + pos % page).repeat_interleave(draft, 0)
        tree = visible_drafts(s["mask"], n, draft, dev) & ((pos >= 0) & (entry >= 0))[:, None]
        slot = torch.cat([slot, own_slot], 1)
        vis = torch.cat([vis, tree.reshape(n * draft, draft)], 1)
    return slot.clamp(min=0), vis[:, None]


def plain_attend(s):
    c = s["case"]
    n, draft, kv, dim = c["batch"], c["draft"], c["kv_heads"], c["dim"]
    group = c["heads"] // kv
    if s["slots"] is None:
        (slot, vis), rows = dense_plan(s), draft
    else:
        (slot, vis), rows = slots_plan(s), 1
    m = slot.shape[0]
    q = s["q"].float().view(m, rows, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(m, kv, rows * group, dim)
    k = rows_of(s, "k", slot).permute(0, 2, 3, 1).contiguous()
    sc = torch.matmul(q, k) * s["scale"]
    see = vis[:, None, :, None].expand(m, kv, rows, group, -1).reshape(m, kv, rows * group, -1)
    sc = torch.where(see, sc, -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(sc - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, rows_of(s, "v", slot).transpose(1, 2).contiguous()) / total
    o = o.view(m, kv, rows, group, dim).transpose(1, 2).reshape(s["q"].shape)
    lse = (torch.log(total) + top).view(m, kv, rows, group).transpose(1, 2).reshape(s["q"].shape[:3])
    return {"out": o.to(s["q"].dtype), "lse": lse}


def plain_prompt(s):
    """The prompts padded to the longest, one KV head after the other (their scores together would be
    as large as the card's memory)."""
    c = s["case"]
    dev, n = s["q"].device, c["batch"]
    kv, dim = c["kv_heads"], c["dim"]
    group = c["heads"] // kv
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    i = torch.arange(c["longest"], device=dev)
    j = torch.arange(c["longest"] + c["context"], device=dev)
    at_q = torch.where(i < lq[:, None], cq[:-1, None] + i, 0)
    at_k = torch.where(j < lk[:, None], ck[:-1, None] + j, 0)
    hide = (j >= lk[:, None])[:, None].expand(n, c["longest"], -1)
    if c["causal"]:
        hide = hide | (j[None, None] > (i[None] + (lk - lq)[:, None])[..., None])
    out = torch.empty(s["q"].shape, device=dev)
    lse = torch.empty(s["q"].shape[:2], device=dev)
    b, t = torch.nonzero(i < lq[:, None], as_tuple=True)
    for h in range(kv):
        heads = slice(h * group, (h + 1) * group)
        q = s["q"][:, heads][at_q].float().transpose(1, 2)
        k = s["k"][:, h][at_k].float().transpose(1, 2).contiguous()[:, None]
        sc = (torch.matmul(q.reshape(n, -1, dim), k[:, 0]) * s["scale"]).view(n, group, c["longest"], -1)
        sc.masked_fill_(hide[:, None], -math.inf)
        top = sc.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        sc.sub_(top).exp_()
        total = sc.sum(-1, keepdim=True)
        o = torch.matmul(sc.view(n, group * c["longest"], -1), s["v"][:, h][at_k].float())
        o = o.view(n, group, c["longest"], dim) / torch.where(total > 0, total, 1.0)
        out[cq[b] + t, heads] = o[b, :, t]
        lse[cq[b] + t, heads] = (torch.log(total) + top)[b, :, t, 0]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"write": plain_write, "read": plain_read, "attend": plain_attend, "prompt": plain_prompt}[op](s)
    import varlen_top_select_amd as vts

    if op == "attend":
        out, lse = vts.tree_attention(
            s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], tree_mask=s["mask"], slots=s["slots"],
            scale=s["scale"], return_lse=True, k_scales=s["k_scales"], v_scales=s["v_scales"])
        return {"out": out, "lse": lse}
    if op == "prompt":
        out, lse = vts.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], cu_seqlens_k=s["cu_k"],
                                        causal=s["case"]["causal"], scale=s["scale"], return_lse=True)
        return {"out": out, "lse": lse}
    if op == "read":
        k, v = vts.read_cache(s["k_cache"], s["v_cache"], s["slots"], k_scales=s["k_scales"],
                              v_scales=s["v_scales"], dtype=DTYPES[s["case"]["dtype"]])
        return {"k": k, "v": v}
    q, k = vts.write_cache(
        s["q"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_scales=s["k_scales"],
        v_scales=s["v_scales"], positions=s["positions"], rotary=s["rotary"],
        interleaved=s["case"]["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6,
        return_k=s["case"]["keep_k"])
    k_cached, v_cached = vts.read_cache(s["k_cache"], s["v_cache"], s["slots"], k_scales=s["k_scales"],
                                        v_scales=s["v_scales"], dtype=s["q"].dtype)
    out = {"q": q, "k_cached": k_cached, "v_cached": v_cached}
    if s["case"]["keep_k"]:
        out["k"] = k
    return out


def work(case):
    kv, dim = case["kv_heads"], case["dim"]
    if case["op"] == "prompt":
        lq, lk = lengths(case), [a + b for a, b in zip(lengths(case), contexts(case))]
        # (the order in which lengths meet contexts is the seed's; the sum of their products is near this)
        pairs = sum(a * b - (a * (a - 1) // 2 if case["causal"] else 0) for a, b in zip(lq, lk))
        rows = 2 * sum(lq) * case["heads"] + 2 * sum(lk) * kv
        return {"bytes": 2 * rows * dim + 4 * sum(lq) * case["heads"], "flops": 4 * dim * case["heads"] * pairs}
    row = row_bytes(case) + (dim // 32 if case["bits"] != 16 else 0)  # of one head
    if case["op"] == "read":
        return {"bytes": 2 * case["slots"] * kv * (row + 2 * dim) + 4 * case["slots"],
                "flops": 2 * case["slots"] * kv * dim}
    if case["op"] == "write":
        n, heads = case["tokens"], case["heads"]
        moved = 2 * dim * (2 * heads + 2 * kv + (kv if case["keep_k"] else 0)) + 4 * case["rot"] + 8
        cached = 2 * kv * (row + row + 2 * dim)  # written, read, returned
        return {"bytes": n * (moved + cached), "flops": 8 * n * (heads + 2 * kv) * dim}
    n, draft, heads = case["batch"], case["draft"], case["heads"]
    qo = 2 * n * draft * heads * dim * 2
    if case["top_k"]:
        seen = sum(min(case["top_k"], x - draft) * draft for x in lengths(case))
        tree = n * draft if case["tree"] else 0
        return {"bytes": 2 * kv * row * (seen + tree) + qo + 4 * seen,
                "flops": 4 * heads * dim * (seen + tree * (draft + 1) // 2)}
    total = sum(lengths(case))
    return {"bytes": 2 * kv * row * total + qo, "flops": 4 * heads * dim * draft * total}


# ---------------------------------------------------------------------------- 64 bits

def grid(bits, dev):
    """Every magnitude of the format in order: an even place has an even mantissa."""
    if bits == 4:
        return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=dev)
    small = [m * 2.0 ** -9 for m in range(8)]
    return torch.tensor(small + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:119],
                        dtype=torch.float64, device=dev)


def through(x, bits):
    """64-bit rows as the format holds them."""
    blocks = x.unflatten(-1, (-1, 32))
    top = blocks.abs().amax(-1, keepdim=True)
    # the least power of two with which the largest stays below 7 (4 bits), or at most at 464 (8)
    part, e = torch.frexp(top / (7 if bits == 4 else 464))
    if bits == 8:
        e = torch.where(part == 0.5, e - 1, e)
    e = torch.where(top == 0, -127, e).clamp(-127, 127)
    unit = torch.exp2(e.double())
    m = blocks.abs() / unit
    numbers = grid(bits, x.device)
    middle = (numbers[1:] + numbers[:-1]) / 2
    below, above = torch.bucketize(m, middle, right=False), torch.bucketize(m, middle, right=True)
    place = torch.where(below % 2 == 0, below, above)  # they differ on a tie alone
    return (numbers[place] * unit * blocks.sign()).flatten(-2)


def exact_write(s):
    c = s["case"]
    dim, rot, bits = c["dim"], c["rot"], c["bits"]
    if rot:
        table = s["rotary"][s["positions"].long()].double()
        turn = torch.complex(table[:, :rot // 2], table[:, rot // 2:])[:, None]

    def form(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / dim + 1e-6).sqrt() * w.double()
        if rot:
            pairs = x[..., :rot]
            pairs = pairs.unflatten(-1, (rot // 2, 2)) if c["interleaved"] else \
                pairs.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
            pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            pairs = pairs if c["interleaved"] else pairs.transpose(-1, -2)
            x = torch.cat([pairs.flatten(-2), x[..., rot:]], -1)
        return x

    k, v = form(s["k"], s["k_norm"]), s["v"].double()
    gone = s["slots"] < 0
    out = {"q": form(s["q"], s["q_norm"])}
    for name, x in (("k_cached", k), ("v_cached", v)):
        x = x.clone() if bits == 16 else through(x, bits)
        x[gone] = 0
        out[name] = x
    if c["keep_k"]:
        out["k"] = k
    return out


def exact_rows(cache, scales, bits, page, slot):
    """64-bit rows of slots, element by element from the format's numbers."""
    data = cache[slot // page, slot % page]
    if bits == 16:
        return data.double()
    if bits == 4:
        data = torch.stack([data % 16, data // 16], -1).flatten(-2)
    sign = torch.where(data >= (8 if bits == 4 else 128), -1.0, 1.0).double()
    size = grid(bits, data.device)[(data % (8 if bits == 4 else 128)).long()]
    power = torch.pow(2.0, scales[slot // page, slot % page].double() - 127)
    return sign * size * power.repeat_interleave(32, -1)


def exact(case, seed):
    """The definitions in 64 bits, request by request."""
    s = prepare(case, seed)
    if case["op"] == "write":
        return exact_write(s)
    if case["op"] == "prompt":
        return exact_prompt(s)
    bits, page = case["bits"], case["page"]
    if case["op"] == "read":
        slot = s["slots"].long()
        return {x: exact_rows(s[x + "_cache"], s[x + "_scales"], bits, page, slot) for x in "kv"}
    draft, kv, dim = case["draft"], case["kv_heads"], case["dim"]
    group = case["heads"] // kv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=out.device)
    for b, length in enumerate(s["lens"].tolist()):
        pos = torch.arange(length, device=out.device)
        home = s["table"][b].long()[pos // page] * page + pos % page
        first = length - draft
        for t in range(draft):
            if s["mask"] is not None:
                bits_of = int(s["mask"][b, t])
                mine = [first + i for i in range(draft) if bits_of >> i & 1]
            else:
                mine = list(range(first, first + t + 1))
            mine = torch.tensor(mine, dtype=torch.long, device=out.device)
            if s["slots"] is not None:
                chosen = s["slots"][b, t].long()
                at = chosen[chosen >= 0]
                if s["mask"] is not None:
                    at = torch.cat([at, home[mine]])
            else:
                at = home[torch.cat([pos[:first], mine])]
            k = exact_rows(s["k_cache"], s["k_scales"], bits, page, at).permute(1, 2, 0).contiguous()
            v = exact_rows(s["v_cache"], s["v_scales"], bits, page, at).transpose(0, 1).contiguous()
            sc = torch.matmul(s["q"][b, t].double().view(kv, group, -1), k) * s["scale"]
            lse[b, t] = torch.logsumexp(sc, -1).view(-1)
            out[b, t] = torch.matmul(torch.softmax(sc, -1), v).view(-1, dim)
    return {"out": out, "lse": lse}


def exact_prompt(s):
    c = s["case"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=out.device)
    group = c["heads"] // c["kv_heads"]
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(c["batch"]):
        q, k, v = s["q"][cq[b]:cq[b + 1]], s["k"][ck[b]:ck[b + 1]], s["v"][ck[b]:ck[b + 1]]
        keep = torch.ones(len(q), len(k), dtype=torch.bool, device=out.device)
        if c["causal"]:
            keep = keep.tril(len(k) - len(q))
        for h in range(c["heads"]):
            sc = q[:, h].double() @ k[:, h // group].double().T.contiguous() * s["scale"]
            sc = torch.where(keep, sc, -math.inf)
            lse[cq[b]:cq[b + 1], h] = torch.logsumexp(sc, -1)
            out[cq[b]:cq[b + 1], h] = torch.softmax(sc, -1) @ v[:, h // group].double()
    return {"out": out, "lse": lse}
