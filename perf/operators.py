"""Cases of the speculative decode step over a paged KV cache.

Four operators, each in a plain form (elementary torch operations in 32 bits, or 64 where whole
numbers depend on long sums) and as a user calls it from ``varlen_top_select_amd``:

  attend   tree_attention        drafted tokens over a paged cache, or over selected slots
  weigh    attention_weight_add  attention weight accumulated per cached entry
  evict    evict_cache           the heaviest entries kept and moved to new pages
  verify   verify_draft          drafted tokens against the target's probabilities
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one request, one token, grouped heads: the smallest decode step, all latency
        dict(name="attend_single", op="attend", batch=1, draft=1, heads=32, kv_heads=8, dim=128,
             page=64, longest=4096, tree=False, top_k=0, dtype="bf16"),
        # a served batch with one drafted token after the real one (next_n 2), ragged lengths
        dict(name="attend_chain", op="attend", batch=64, draft=2, heads=64, kv_heads=8, dim=128,
             page=64, longest=16384, tree=False, top_k=0, dtype="bf16"),
        # a tree of 16 drafted tokens over long contexts: many query rows per cached row
        dict(name="attend_tree_long", op="attend", batch=8, draft=16, heads=64, kv_heads=8,
             dim=128, page=64, longest=65536, tree=True, top_k=0, dtype="bf16"),
        # each drafted row attends the 2048 slots that the selection gave it, and its ancestors
        dict(name="attend_slots", op="attend", batch=64, draft=2, heads=64, kv_heads=4, dim=128,
             page=64, longest=65536, tree=True, top_k=2048, dtype="bf16"),
        # odd everything: 7 heads a group, 5 drafted tokens, pages of 24, head size 64, fp16
        dict(name="attend_odd", op="attend", batch=13, draft=5, heads=14, kv_heads=2, dim=64,
             page=24, longest=9001, tree=True, top_k=0, dtype="fp16"),
        # the weights of one served batch's step, after attend_chain
        dict(name="weigh_chain", op="weigh", batch=64, draft=2, heads=64, kv_heads=8, dim=128,
             page=64, longest=16384, tree=False, top_k=0, dtype="bf16"),
        # a small batch with a tree, only the accepted rows count
        dict(name="weigh_tree", op="weigh", batch=3, draft=7, heads=12, kv_heads=4, dim=64,
             page=16, longest=2500, tree=True, top_k=0, dtype="fp16"),
        # a batch cut back from about 8192 entries to 4096
        dict(name="evict_half", op="evict", batch=32, kv_heads=8, dim=128, page=64, longest=8192,
             keep=4096, sinks=4, recent=512, dtype="bf16"),
        # one request a page over its budget
        dict(name="evict_page", op="evict", batch=1, kv_heads=8, dim=128, page=64, longest=1088,
             keep=1024, sinks=4, recent=64, dtype="bf16"),
        # a served batch, three tokens drawn from a draft model's distributions
        dict(name="verify_chain", op="verify", batch=64, draft=3, vocab=131072, branch=1,
             drawn=True, dtype="fp32"),
        # trees of 24 tokens, up to three siblings a node, drawn, 16-bit probabilities
        dict(name="verify_tree", op="verify", batch=16, draft=24, vocab=100003, branch=3,
             drawn=True, dtype="bf16"),
        # one request whose drafted token was chosen and not drawn: latency
        dict(name="verify_single", op="verify", batch=1, draft=1, vocab=32768, branch=1,
             drawn=False, dtype="fp32"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attend", "attend", "weigh", "evict", "verify"])
    if op == "verify":
        batch = log(1, 64)
        return dict(op=op, batch=batch, draft=rng.randint(1, 24 if batch <= 16 else 3),
                    vocab=log(1000, 131072), branch=rng.randint(1, 3),
                    drawn=rng.random() < 0.7, dtype=rng.choice(["fp32", "bf16", "fp16"]))
    page = rng.choice([1, 16, 24, 64, 64, 128])
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "evict":
        longest = log(200, 8192)
        keep = max(8, int(longest * rng.uniform(0.3, 0.95)))
        return dict(op=op, batch=log(1, 32), kv_heads=kv_heads, dim=dim, page=page,
                    longest=longest, keep=keep, sinks=rng.randint(0, 4),
                    recent=rng.randint(0, keep // 4), dtype=dtype)
    batch = log(1, 64)
    group = rng.choice([1, 3, 4, 7, 8, 16])
    longest = min(log(100, 65536), 16384 * 64 // batch)
    draft = rng.randint(1, 16 if batch <= 8 else 4)
    while draft * group * kv_heads > 1024 // (1 if batch <= 8 else 8):
        group = max(1, group // 2)
        draft = max(1, draft - 1)
    top_k = log(64, 2048) if op == "attend" and rng.random() < 0.35 else 0
    return dict(op=op, batch=batch, draft=draft, heads=group * kv_heads, kv_heads=kv_heads,
                dim=dim, page=page, longest=longest, tree=rng.random() < 0.6, top_k=top_k,
                dtype=dtype)


# ---------------------------------------------------------------------------- inputs

def lengths(case):
    """The batch's lengths, spread over [longest / 3, longest]; the seed only changes their order."""
    n, hi = case["batch"], case["longest"]
    lo = max(case.get("draft", 1), hi // 3)
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


def random_parents(n, draft, branch, gen, dev):
    """Trees in level order of about `branch` siblings a node; some nodes hang from another level."""
    node = torch.arange(draft, device=dev)
    if branch == 1:
        return (node - 1).repeat(n, 1).to(torch.int32)
    top = node // branch
    low = torch.clamp(top - 1, min=0)
    pick = torch.rand(n, draft, generator=gen, device=dev)
    half = low + (pick * (top - low + 1)).long().clamp(max=top - low)
    parent = torch.where(node[None] % 5 == 4, half, top[None].expand(n, -1)) - 1
    return torch.minimum(parent, node[None] - 1).to(torch.int32)


def ancestor_bits(parents):
    """Each node's ancestors and itself as bits of an int64."""
    n, draft = parents.shape
    bits = torch.zeros(n, draft, dtype=torch.int64, device=parents.device)
    for t in range(draft):
        p = parents[:, t].long()
        up = bits.gather(1, p.clamp(min=0)[:, None])[:, 0]
        bits[:, t] = torch.where(p >= 0, up, 0) | (1 << t)
    return bits


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    n = case["batch"]
    s = {"case": case}
    if case["op"] == "verify":
        draft, vocab = case["draft"], case["vocab"]

        def normal(*shape):
            return torch.randn(*shape, generator=gen, device=dev)

        base = 4.0 * normal(n, draft + 1, vocab)
        s["target"] = torch.softmax(base, -1).to(dtype)
        near = torch.softmax(base[:, :draft] + 0.7 * normal(n, draft, vocab), -1)
        s["parents"] = random_parents(n, draft, case["branch"], gen, dev)
        row = (s["parents"].long() + 1)
        near_row = near.gather(1, row[:, :, None].expand(-1, -1, vocab))
        if case["drawn"]:
            cdf = torch.cumsum(near_row.double(), -1)
            pick = torch.rand(n, draft, 1, generator=gen, device=dev, dtype=torch.float64)
            tokens = torch.searchsorted(cdf, pick * cdf[..., -1:]).clamp(max=vocab - 1)
        else:  # siblings are their parent's best tokens, in order
            node = torch.arange(draft, device=dev)
            elder = (row[:, :, None] == row[:, None]) & (node[None] < node[:, None])
            best = torch.topk(near_row, min(draft, vocab), dim=-1).indices
            tokens = best.gather(2, elder.sum(-1)[..., None])
        s["tokens"] = tokens[..., 0].to(torch.int32).contiguous()
        s["draft"] = near.to(dtype) if case["drawn"] else None
        s["uniforms"] = torch.rand(n, draft + 1, generator=gen, device=dev)
        if case["branch"] == 1:
            s["parents"] = None
        return s

    heads_kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    s["lens"], s["table"], pool = paged(case, gen, dev)

    def cache():
        return torch.randn(pool, page, heads_kv, dim, generator=gen, device=dev, dtype=dtype)

    s["k"] = cache()
    if case["op"] == "evict":
        s["v"] = cache()
        # accumulated weights fall off steeply, with many entries that never mattered
        u = torch.rand(n, heads_kv, case["longest"], generator=gen, device=dev)
        s["weights"] = torch.where(u < 0.1, 0.0, u.pow(8) * 3)
        pages = -(-case["keep"] // page)
        s["k_out"] = torch.zeros(n * pages, page, heads_kv, dim, device=dev, dtype=dtype)
        s["v_out"] = torch.zeros_like(s["k_out"])
        order = torch.randperm(n * pages, generator=gen, device=dev)
        s["out_table"] = order.view(n, pages).to(torch.int32).contiguous()
        return s

    draft, heads = case["draft"], case["heads"]
    s["q"] = (1.5 * torch.randn(n, draft, heads, dim, generator=gen, device=dev)).to(dtype)
    s["scale"] = 1.0 / math.sqrt(dim)
    s["mask"] = None
    if case["tree"]:
        s["mask"] = ancestor_bits(random_parents(n, draft, 3, gen, dev))
    s["slots"] = None
    if case["op"] == "attend":
        s["v"] = cache()
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
    s["weights"] = torch.rand(n, heads_kv, case["longest"], generator=gen, device=dev)
    s["keep_rows"] = (torch.rand(n, draft, generator=gen, device=dev) < 0.7) if case["tree"] else None
    s["lse"] = dense_lse(s)
    return s


# ---------------------------------------------------------------------------- plain forms

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
    first = (lens - draft)[:, None]
    i = pos[None] - first
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


def rows_of(cache, slot):
    """fp32 cache rows of [n, S] slots as [n, Hkv, S, D]."""
    flat = cache.view(-1, cache.shape[2], cache.shape[3])
    return flat[slot].permute(0, 2, 1, 3).float()


def scores(q, cache, slot, vis, scale):
    """Scores [n, Hkv, rows * G, S], -inf where masked; q is [n, rows, Hq, D]."""
    n, rows, heads, dim = q.shape
    kv = cache.shape[2]
    group = heads // kv
    qr = q.float().view(n, rows, kv, group, dim).permute(0, 2, 1, 3, 4)
    k = rows_of(cache, slot).transpose(2, 3).contiguous()
    sc = torch.matmul(qr.reshape(n, kv, rows * group, dim), k) * scale
    see = vis[:, None, :, None].expand(n, kv, rows, group, -1).reshape(n, kv, rows * group, -1)
    return torch.where(see, sc, -math.inf)


def softmax_parts(sc):
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(sc - top)
    return e, e.sum(-1, keepdim=True), top


def ungroup(x, n, rows, kv):
    """[n, kv, rows * G, ...] to [n, rows, kv * G, ...]."""
    group = x.shape[2] // rows
    x = x.view(n, kv, rows, group, *x.shape[3:])
    return x.transpose(1, 2).reshape(n, rows, kv * group, *x.shape[4:])


def dense_lse(s):
    slot, vis = dense_plan(s)
    e, total, top = softmax_parts(scores(s["q"], s["k"], slot, vis, s["scale"]))
    n, draft = s["case"]["batch"], s["case"]["draft"]
    return ungroup((torch.log(total) + top)[..., 0], n, draft, s["case"]["kv_heads"]).contiguous()


def plain_attend(s):
    n, draft, kv = s["case"]["batch"], s["case"]["draft"], s["case"]["kv_heads"]
    q = s["q"]
    if s["slots"] is None:
        slot, vis = dense_plan(s)
        rows = draft
    else:
        slot, vis = slots_plan(s)
        q = q.view(n * draft, 1, *q.shape[2:])
        rows = 1
    e, total, top = softmax_parts(scores(q, s["k"], slot, vis, s["scale"]))
    v = torch.where(vis.any(1)[:, None, :, None], rows_of(s["v"], slot), 0.0)
    o = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)
    m = q.shape[0]
    o = ungroup(o, m, rows, kv).view(s["q"].shape).to(s["q"].dtype)
    lse = ungroup((torch.log(total) + top)[..., 0], m, rows, kv).view(s["q"].shape[:3])
    return {"out": o, "lse": lse}


def plain_weigh(s):
    n, draft, kv = s["case"]["batch"], s["case"]["draft"], s["case"]["kv_heads"]
    slot, vis = dense_plan(s)
    sc = scores(s["q"], s["k"], slot, vis, s["scale"])
    group = s["q"].shape[2] // kv
    lse = s["lse"].view(n, draft, kv, group).transpose(1, 2).reshape(n, kv, -1, 1)
    p = torch.where(lse > -math.inf, torch.exp(sc - lse), 0.0)
    if s["keep_rows"] is not None:
        take = s["keep_rows"][:, None, :, None].expand(n, kv, draft, group).reshape(n, kv, -1, 1)
        p = torch.where(take, p, 0.0)
    s["weights"] += p.sum(2)
    return s["weights"]


def plain_evict(s):
    c = s["case"]
    n, kv, page, keep = c["batch"], c["kv_heads"], c["page"], c["keep"]
    dev = s["k"].device
    pos = torch.arange(c["longest"], device=dev)
    lens = s["lens"].long()[:, None, None]
    live = (pos < lens).expand(n, kv, -1)
    safe = live & ((pos < c["sinks"]) | (pos >= lens - c["recent"]))
    rank = torch.where(safe, math.inf, torch.where(live, s["weights"], -math.inf))
    order = torch.argsort(rank, dim=-1, descending=True, stable=True)[..., :keep]
    count = torch.clamp(s["lens"].long(), max=keep)
    slot_of = torch.arange(keep, device=dev)
    short = slot_of[: order.shape[-1]] >= count[:, None, None]
    order = torch.sort(torch.where(short, c["longest"], order), dim=-1).values
    if order.shape[-1] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=c["longest"])
    full = slot_of[None, None] < count[:, None, None]
    at = torch.where(full, order, 0)
    w = torch.where(full, s["weights"].gather(2, at), 0.0)
    entry = s["table"].long()[:, None].expand(n, kv, -1).gather(2, at // page)
    src = entry * page + at % page
    dst = (s["out_table"].long()[:, slot_of // page] * page + slot_of % page)[:, None].expand(n, kv, -1)
    head = torch.arange(kv, device=dev)[None, :, None].expand_as(src)
    src, dst, head = src[full.expand_as(src)], dst[full.expand_as(src)], head[full.expand_as(src)]
    dim = c["dim"]
    s["k_out"].view(-1, kv, dim)[dst, head] = s["k"].view(-1, kv, dim)[src, head]
    s["v_out"].view(-1, kv, dim)[dst, head] = s["v"].view(-1, kv, dim)[src, head]
    kept = torch.where(full, order, -1).to(torch.int32)
    return {"kept": kept, "lens": count.to(torch.int32), "weights": w, "k": s["k_out"], "v": s["v_out"]}


def plain_verify(s):
    """One step per drafted node, all requests at once; sums over the vocabulary in 64 bits."""
    target, q_all, u = s["target"], s["draft"], s["uniforms"].double()
    n, draft = s["tokens"].shape
    vocab, dev = target.shape[2], target.device
    each = torch.arange(n, device=dev)
    parents = s["parents"]
    if parents is None:
        parents = (torch.arange(draft, device=dev) - 1).expand(n, -1)
    cur = torch.full((n,), -1, device=dev)
    a = torch.zeros(n, dtype=torch.float64, device=dev)
    mass = torch.ones_like(a)
    gone = torch.zeros(n, vocab, dtype=torch.bool, device=dev)
    path = torch.full((n, draft), -1, device=dev)
    count = torch.zeros(n, dtype=torch.int64, device=dev)

    def residual():
        p = target[each, cur + 1].double()
        if q_all is None:
            return torch.where(gone, 0.0, p)
        q = q_all[each, (cur + 1).clamp(max=draft - 1)].double()
        return torch.clamp(p - a[:, None] * torch.where(a[:, None] > 0, q, 0.0), min=0)

    for t in range(draft):
        x = s["tokens"][:, t].long()
        here = parents[:, t] == cur
        p = target[each, cur + 1, x].double()
        if q_all is None:
            r, bar = torch.where(gone[each, x], 0.0, p), u[:, t] * mass
        else:
            q = q_all[each, (cur + 1).clamp(max=draft - 1), x].double()
            r, bar = torch.clamp(p - a * q, min=0), u[:, t] * q * mass
        yes, no = here & (bar < r), here & ~(bar < r)
        path[each, count.clamp(max=draft - 1)] = torch.where(
            yes, t, path[each, count.clamp(max=draft - 1)])
        count += yes
        cur = torch.where(yes, t, cur)
        if q_all is None:
            mass = torch.where(no, mass - torch.where(gone[each, x], 0.0, p), mass)
            gone[each, x] |= no
            gone &= ~yes[:, None]
        else:
            a = torch.where(no, a + mass, a)
            mass = torch.where(no, residual().sum(-1), mass)
        a, mass = torch.where(yes, 0.0, a), torch.where(yes, 1.0, mass)
    r = residual()
    some = r.sum(-1, keepdim=True) > 0
    r = torch.where(some, r, target[each, cur + 1].double())
    cdf = torch.cumsum(r, -1)
    token = (cdf > u[:, draft:] * cdf[:, -1:]).int().argmax(-1)
    return {"path": path.to(torch.int32), "count": count.to(torch.int32),
            "token": token.to(torch.int32)}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"attend": plain_attend, "weigh": plain_weigh, "evict": plain_evict,
                "verify": plain_verify}[op](s)
    import varlen_top_select_amd as vts

    if op == "attend":
        out, lse = vts.tree_attention(s["q"], s["k"], s["v"], s["table"], s["lens"],
                                      tree_mask=s["mask"], slots=s["slots"], scale=s["scale"],
                                      return_lse=True)
        return {"out": out, "lse": lse}
    if op == "weigh":
        return vts.attention_weight_add(s["weights"], s["q"], s["k"], s["table"], s["lens"],
                                        s["lse"], tree_mask=s["mask"], row_keep=s["keep_rows"],
                                        scale=s["scale"])
    if op == "evict":
        c = s["case"]
        kept, lens, weights = vts.evict_cache(
            s["weights"], s["k"], s["v"], s["table"], s["lens"], c["keep"], s["k_out"], s["v_out"],
            s["out_table"], sinks=c["sinks"], recent=c["recent"])
        return {"kept": kept, "lens": lens, "weights": weights, "k": s["k_out"], "v": s["v_out"]}
    path, count, token = vts.verify_draft(s["target"], s["tokens"], s["uniforms"],
                                          draft_probs=s["draft"], parents=s["parents"])
    return {"path": path, "count": count, "token": token}


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    n = case["batch"]
    if case["op"] == "verify":
        rows = 2 if case["drawn"] else 1
        total = n * rows * case["vocab"]
        return {"bytes": total * size + n * case["draft"] * 64, "flops": 3 * total}
    lens = lengths(case)
    row = case["kv_heads"] * case["dim"] * size
    if case["op"] == "evict":
        kept = sum(min(x, case["keep"]) for x in lens)
        w = 4 * case["kv_heads"]
        return {"bytes": 4 * kept * row + sum(lens) * w + kept * 2 * w, "flops": sum(lens) * case["kv_heads"]}
    draft, qo = case["draft"], n * case["draft"] * case["heads"] * case["dim"] * size
    lanes = case["heads"] * case["dim"]
    if case["top_k"]:
        seen = sum(min(case["top_k"], x - draft) * draft for x in lens)
        tree = n * draft * (draft + 1) // 2 if case["tree"] else 0
        return {"bytes": 2 * row * (seen + (n * draft if case["tree"] else 0)) + 2 * qo + 4 * seen,
                "flops": 4 * lanes * (seen + tree)}
    total = sum(lens)
    if case["op"] == "attend":
        return {"bytes": 2 * row * total + 2 * qo, "flops": 4 * lanes * draft * total}
    return {"bytes": row * total + qo + 8 * case["kv_heads"] * total, "flops": 2 * lanes * draft * total}


# ---------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definitions, request by request, in 64 bits; whole-number outputs of a draw included."""
    s = prepare(case, seed)
    if case["op"] == "verify":
        return exact_verify(s)
    if case["op"] == "evict":
        return exact_evict(s)
    page, draft, kv = case["page"], case["draft"], case["kv_heads"]
    group = case["heads"] // kv
    flat_k = s["k"].view(-1, kv, case["dim"])
    flat_v = s["v"].view(-1, kv, case["dim"]) if "v" in s else None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=out.device)
    weights = s["weights"].double() if case["op"] == "weigh" else None
    for b, length in enumerate(s["lens"].tolist()):
        pos = torch.arange(length, device=out.device)
        home = s["table"][b].long()[pos // page] * page + pos % page
        first = length - draft
        for t in range(draft):
            if s["mask"] is not None:
                bits = int(s["mask"][b, t])
                mine = [first + i for i in range(draft) if bits >> i & 1]
            else:
                mine = list(range(first, first + t + 1))
            mine = torch.tensor(mine, dtype=torch.long, device=out.device)
            if s["slots"] is not None:
                chosen = s["slots"][b, t].long()
                at = chosen[chosen >= 0]
                if s["mask"] is not None:
                    at = torch.cat([at, home[mine]])
            else:
                seen = torch.cat([pos[:first], mine])
                at = home[seen]
            k = flat_k[at].double().permute(1, 2, 0).contiguous()
            q = s["q"][b, t].double().view(kv, group, -1)
            sc = torch.matmul(q, k) * s["scale"]
            if weights is not None:
                if s["keep_rows"] is None or bool(s["keep_rows"][b, t]):
                    weights[b, :, seen] += torch.exp(sc - s["lse"][b, t].double().view(kv, group, 1)).sum(1)
                continue
            lse[b, t] = torch.logsumexp(sc, -1).view(-1)
            p = torch.softmax(sc, -1)
            out[b, t] = torch.matmul(p, flat_v[at].double().transpose(0, 1).contiguous()).view(-1, case["dim"])
    return weights if weights is not None else {"out": out, "lse": lse}


def exact_evict(s):
    """Only the copies come out of this as numbers: values moved, none computed."""
    c = s["case"]
    page, keep = c["page"], c["keep"]
    kept = torch.full((c["batch"], c["kv_heads"], keep), -1, dtype=torch.int32)
    moved = torch.zeros(c["batch"], c["kv_heads"], keep, dtype=torch.float64)
    k_out, v_out = s["k_out"].double(), s["v_out"].double()
    lens = s["lens"].tolist()
    weights = s["weights"].cpu()
    for b, length in enumerate(lens):
        for h in range(c["kv_heads"]):
            w = weights[b, h, :length].tolist()
            middle = range(min(c["sinks"], length), max(min(c["sinks"], length), length - c["recent"]))
            safe = [j for j in range(length) if j < c["sinks"] or j >= length - c["recent"]]
            best = sorted(middle, key=lambda j: (-w[j], j))[: max(0, keep - len(safe))]
            take = torch.tensor(sorted(safe + best)[:keep] if length > keep else list(range(length)))
            kept[b, h, : len(take)] = take.int()
            moved[b, h, : len(take)] = weights[b, h][take].double()
            take = take.to(k_out.device)
            i = torch.arange(len(take), device=k_out.device)
            src, dst = s["table"][b].long()[take // page], s["out_table"][b].long()[i // page]
            k_out[dst, i % page, h] = s["k"][src, take % page, h].double()
            v_out[dst, i % page, h] = s["v"][src, take % page, h].double()
    count = torch.tensor([min(x, keep) for x in lens], dtype=torch.int32)
    return {"kept": kept, "lens": count, "weights": moved, "k": k_out, "v": v_out}


def exact_verify(s):
    """Residuals formed one after the other, each normalised, as the rule is stated."""
    n, draft = s["tokens"].shape
    path = torch.full((n, draft), -1, dtype=torch.int32)
    counts, tokens = [], []
    drafted, u = s["tokens"].tolist(), s["uniforms"].double().tolist()
    parents = s["parents"].tolist() if s["parents"] is not None else [list(range(-1, draft - 1))] * n
    for b in range(n):
        cur, steps, dist = -1, 0, s["target"][b, 0].double()
        for t in range(draft):
            if parents[b][t] != cur:
                continue
            x = drafted[b][t]
            if s["draft"] is None:
                q = torch.zeros_like(dist)
                q[x] = 1.0
            else:
                q = s["draft"][b, cur + 1].double()
            if u[b][t] * float(q[x]) < float(dist[x]):
                path[b, steps] = t
                steps, cur = steps + 1, t
                dist = s["target"][b, t + 1].double()
                continue
            rest = torch.clamp(dist - q, min=0)
            dist = rest / rest.sum() if float(rest.sum()) > 0 else rest
        if float(dist.sum()) == 0:
            dist = s["target"][b, cur + 1].double()
        cdf = torch.cumsum(dist, 0)
        counts.append(steps)
        tokens.append(int((cdf > u[b][draft] * float(cdf[-1])).int().argmax()))
    return {"path": path, "count": torch.tensor(counts, dtype=torch.int32),
            "token": torch.tensor(tokens, dtype=torch.int32)}
