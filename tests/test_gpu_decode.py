"""The decode-step operators against plain 64-bit forms (tests/decode_ref.py):
lengths from zero on, odd pages and groups, masks that leave rows empty, entries
that are not there, infinities and NaN in places that are not seen, strided
caches, slot lists, streams, graphs, workspaces shared between shapes."""
import math

import numpy as np
import pytest
import torch

import varlen_top_select_amd as vts
from tests import decode_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

DEV = "cuda"


def say(*a):
    print(*a, flush=True)


def make_cache(gen, lens, page, kv, dim, dtype, extra_width=1, order=None):
    """K and V of random values, a table with pages in random order, -1 past the end."""
    used = [-(-max(x, 0) // page) for x in lens]
    width = max(used + [1]) + extra_width
    pool = sum(used) + 2
    perm = torch.randperm(pool, generator=gen)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(used):
        table[b, :m] = perm[at:at + m].int()
        at += m
    shape = (pool, page, kv, dim)
    k, v = (torch.randn(shape, generator=gen).to(dtype).to(DEV) for _ in range(2))
    if order == "heads_first":  # [pages, kv, page, dim] seen as [pages, page, kv, dim]
        k, v = (x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (k, v))
    elif order == "padded":
        wide = [torch.zeros(pool, page, kv + 1, dim + 16, dtype=dtype, device=DEV) for _ in range(2)]
        for w, x in zip(wide, (k, v)):
            w[:, :, :kv, :dim] = x
        k, v = (w[:, :, :kv, :dim] for w in wide)
    return k, v, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def random_mask(gen, batch, draft):
    parents = torch.stack([torch.cat([torch.tensor([-1])] + [
        torch.randint(-1, t, (1,), generator=gen) for t in range(1, draft)]) for _ in range(batch)])
    return vts.tree_mask_from_parents(parents.int()).to(DEV), parents.int()


def check_attend(q, k, v, table, lens, mask=None, slots=None, scale=None, **kw):
    out, lse = vts.tree_attention(q, k, v, table, lens, tree_mask=mask, slots=slots, scale=scale,
                                  return_lse=True, **kw)
    torch.cuda.synchronize()
    o64, l64, mag, reach = ref.attend(q, k, v, table, lens, mask, slots, scale)
    count = (0 if slots is None else slots.shape[-1]) + int(lens.clamp(min=0).max()) + 1
    ob, lb = ref.attend_bounds(o64, mag, reach, count, q.shape[3], q.dtype)
    got, gl = out.cpu().double(), lse.cpu().double()
    empty = l64 == -math.inf
    assert torch.equal(gl == -math.inf, empty)
    assert (got[empty] == 0).all()
    worst = ((got - o64).abs() / ob).max().item()
    assert worst <= 1, f"output {worst:.3g} times its bound"
    worst = ((gl - l64).abs()[~empty] / lb[~empty]).max().item() if (~empty).any() else 0
    assert worst <= 1, f"lse {worst:.3g} times its bound"
    return out, lse


CASES = [
    # batch lengths, draft, heads, kv, dim, page, tree, dtype
    ([1], 1, 1, 1, 64, 16, False, torch.bfloat16),
    ([0, 1, 2, 31, 32, 33], 1, 8, 2, 128, 16, False, torch.bfloat16),
    ([0, 1, 2, 3, 4, 5, 127, 128, 129, 130], 3, 6, 3, 64, 1, False, torch.float16),
    ([5, 300, 7, 1000], 5, 14, 2, 64, 24, True, torch.float16),
    ([64, 65, 63, 700], 4, 32, 8, 128, 64, True, torch.bfloat16),
    ([200, 90], 7, 24, 2, 128, 7, True, torch.bfloat16),      # 84 rows: two row blocks
    ([150, 64, 40], 64, 4, 2, 64, 16, True, torch.bfloat16),  # 64 drafted tokens, a length below
    ([2500], 2, 16, 1, 128, 128, False, torch.float16),       # one list over many workgroups
    ([777, 1, 300], 1, 40, 1, 128, 32, False, torch.bfloat16),  # 40 rows of one token
    # four heads or a multiple: a head to a wave
    ([2600, 33, 0, 1], 3, 32, 4, 64, 16, True, torch.bfloat16),
    ([1100, 2, 31, 65], 2, 48, 4, 128, 24, True, torch.float16),
    ([4000], 1, 8, 8, 128, 64, False, torch.bfloat16),
    ([130, 0, 5000], 2, 12, 12, 64, 1, False, torch.float16),
    ([500, 90], 9, 32, 8, 128, 16, True, torch.bfloat16),  # 36 rows: not a head to a wave
    ([(x * 61) % 300 for x in range(16)] + [4000] * 16, 1, 16, 4, 64, 16, False, torch.bfloat16),
    ([100] * 31 + [9000], 2, 16, 4, 128, 32, True, torch.float16),  # one list over most workgroups
    ([20000], 1, 2, 1, 64, 64, False, torch.bfloat16),  # blocks of parts
    # wide: 64, 128 rows and more to a KV head, lists that end anywhere
    ([1, 0, 63, 64, 65, 129, 700], 16, 8, 2, 128, 16, True, torch.bfloat16),
    ([3000, 17], 20, 12, 2, 64, 24, True, torch.float16),
    ([1500, 129, 64], 40, 8, 2, 128, 32, True, torch.float16),
    ([900, 70], 64, 10, 2, 64, 64, False, torch.bfloat16),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_attend_paged(i):
    lens, draft, heads, kv, dim, page, tree, dtype = CASES[i]
    say("attend", CASES[i])
    gen = torch.Generator().manual_seed(100 + i)
    k, v, table, n = make_cache(gen, lens, page, kv, dim, dtype)
    q = (1.5 * torch.randn(len(lens), draft, heads, dim, generator=gen)).to(dtype).to(DEV)
    mask = random_mask(gen, len(lens), draft)[0] if tree else None
    check_attend(q, k, v, table, n, mask)


@pytest.mark.parametrize("order", ["heads_first", "padded"])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_strides(order, dim):
    gen = torch.Generator().manual_seed(7)
    k, v, table, n = make_cache(gen, [70, 200, 33], 16, 3, dim, torch.bfloat16, order=order)
    assert not k.is_contiguous()
    # q as [batch, heads, draft, dim] seen the other way round, the table as a slice
    q = torch.randn(3, 6, 2, dim, generator=gen).bfloat16().to(DEV).transpose(1, 2)
    wide = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    wide[:, : table.shape[1]] = table
    check_attend(q, k, v, wide[:, : table.shape[1]], n)


def test_attend_scales():
    gen = torch.Generator().manual_seed(8)
    k, v, table, n = make_cache(gen, [150, 300], 16, 2, 64, torch.bfloat16)
    q = torch.randn(2, 2, 4, 64, generator=gen).bfloat16().to(DEV)
    for scale in (0.0, -0.3, 2.0):  # sharp, uniform and reversed softmax
        check_attend(q, k, v, table, n, scale=scale)


def test_attend_rising_scores():
    """Scores that climb along the cache, so the running maximum keeps moving."""
    gen = torch.Generator().manual_seed(9)
    k, v, table, n = make_cache(gen, [1500], 16, 1, 64, torch.float16)
    order = table[0, : -(-1500 // 16)].long()
    ramp = torch.linspace(0, 20, order.numel() * 16, device=DEV).view(-1, 16, 1)
    k[order, :, :, 0] = ramp.half()
    q = torch.zeros(1, 1, 16, 64, dtype=torch.float16, device=DEV)
    q[..., 0] = 4
    q[..., 1] = 0.5
    check_attend(q, k, v, table, n, scale=1.0)


def test_attend_entries_not_there():
    gen = torch.Generator().manual_seed(10)
    k, v, table, n = make_cache(gen, [100, 100, 40], 16, 2, 64, torch.bfloat16)
    table[0, 2] = -1
    table[0, 4] = k.shape[0]          # one past the last page
    table[1, :] = 2 ** 31 - 1         # nothing of this request is there
    n[2] = 10 ** 9                    # longer than its table row
    table[2, 3:] = -7
    q = torch.randn(3, 3, 4, 64, generator=gen).bfloat16().to(DEV)
    out, lse = check_attend(q, k, v, table, n)
    assert (lse[1] == -math.inf).all() and (out[1] == 0).all()
    n[2] = -5
    check_attend(q, k, v, table, n)


def test_attend_empty_mask_rows():
    gen = torch.Generator().manual_seed(11)
    k, v, table, n = make_cache(gen, [4, 60], 16, 2, 64, torch.bfloat16)
    q = torch.randn(2, 4, 4, 64, generator=gen).bfloat16().to(DEV)
    mask = torch.tensor([[0, 1, 0, 15], [0, 0, 8, 5]], dtype=torch.int64, device=DEV)
    out, lse = check_attend(q, k, v, table, n, mask)
    assert (out[0, 0] == 0).all() and (out[0, 2] == 0).all()
    assert (lse[0, 0] == -math.inf).all()
    mask[0] = -1  # every bit, those past the drafted tokens among them
    check_attend(q, k, v, table, n, mask)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype,heads", [(torch.bfloat16, 4), (torch.float16, 4),
                                         (torch.bfloat16, 16), (torch.float16, 40)])
def test_attend_unseen_infinities(bad, dtype, heads):
    """Values of unseen places (past the length, unused pages, drafted tokens of
    other branches) do not reach a row, whatever they are."""
    gen = torch.Generator().manual_seed(12)
    lens, page, draft = [70, 21, 5], 16, 5
    k, v, table, n = make_cache(gen, lens, page, 2, 128, dtype)
    q = torch.randn(3, draft, heads, 128, generator=gen).to(dtype).to(DEV)
    mask = torch.tensor([[1, 2, 4, 9, 0]] * 3, dtype=torch.int64, device=DEV)
    clean, clean_lse = vts.tree_attention(q, k, v, table, n, tree_mask=mask, return_lse=True)
    live = torch.zeros(k.shape[0], page, dtype=torch.bool, device=DEV)
    for b, m in enumerate(lens):
        for pos in range(m):
            live[table[b, pos // page].long(), pos % page] = True
    k2, v2 = k.clone(), v.clone()
    k2[~live], v2[~live] = bad, bad
    out, lse = vts.tree_attention(q, k2, v2, table, n, tree_mask=mask, return_lse=True)
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
    for b, m in enumerate(lens):  # drafted token 4 is seen by no row, token 1 by row 1 alone
        pos = m - draft + 4
        k2[table[b, pos // page].long(), pos % page] = bad
        v2[table[b, pos // page].long(), pos % page] = bad
    out, lse = vts.tree_attention(q, k2, v2, table, n, tree_mask=mask, return_lse=True)
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
    for b, m in enumerate(lens):
        pos = m - draft + 1
        v2[table[b, pos // page].long(), pos % page, :, 3] = bad
    out, lse = vts.tree_attention(q, k2, v2, table, n, tree_mask=mask, return_lse=True)
    others = [0, 2, 3, 4]
    assert torch.equal(out[:, others], clean[:, others]) and torch.equal(lse, clean_lse)
    want = out[:, 1, :, 3].float()
    assert (want.isnan() if math.isnan(bad) else want == bad).all()
    keep = [c for c in range(128) if c != 3]
    assert torch.equal(out[:, 1][:, :, keep], clean[:, 1][:, :, keep])


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("page,dim,top_k", [(16, 128, 50), (24, 64, 200), (64, 128, 129)])
def test_attend_slots(tree, page, dim, top_k):
    gen = torch.Generator().manual_seed(13 + top_k)
    lens, draft = [300, 5, 120], 3
    k, v, table, n = make_cache(gen, lens, page, 2, dim, torch.bfloat16)
    q = torch.randn(3, draft, 10, dim, generator=gen).bfloat16().to(DEV)
    slots = torch.randint(-1, k.shape[0] * page, (3, draft, top_k), generator=gen, dtype=torch.int32)
    slots[0, 1, top_k // 2:] = -1
    slots[1, 0] = -1                                    # a row without slots
    slots[2, 2, ::7] = k.shape[0] * page                # past the cache
    slots[2, 1, 0] = -2 ** 31
    mask = random_mask(gen, 3, draft)[0] if tree else None
    check_attend(q, k, v, table, n, mask, slots.to(DEV))


@pytest.mark.parametrize("heads,dim,dtype", [(40, 128, torch.bfloat16), (80, 64, torch.float16),
                                             (150, 64, torch.bfloat16)])
def test_attend_slots_of_many_heads(heads, dim, dtype):
    gen = torch.Generator().manual_seed(15 + heads)
    k, v, table, n = make_cache(gen, [300, 5], 16, 1, dim, dtype)
    q = torch.randn(2, 2, heads, dim, generator=gen).to(dtype).to(DEV)
    slots = torch.randint(-1, k.shape[0] * 16, (2, 2, 150), generator=gen, dtype=torch.int32)
    slots[1, 0] = -1
    check_attend(q, k, v, table, n, random_mask(gen, 2, 2)[0], slots.to(DEV))
    check_attend(q, k, v, table, n, None, slots.to(DEV))


def test_attend_slots_of_the_selection():
    """The slots are what topk_page_table_transform writes."""
    gen = torch.Generator().manual_seed(17)
    lens, draft, page, top_k = [400, 90], 2, 16, 64
    k, v, table, n = make_cache(gen, lens, page, 2, 128, torch.bfloat16)
    width = table.shape[1] * page
    scores = torch.randn(2 * draft, width, generator=gen).to(DEV)
    prefix = (n - draft).repeat_interleave(draft).contiguous()
    rows = table.repeat_interleave(draft, 0).contiguous()
    slots, _ = vts.topk_page_table_transform(scores, prefix, rows, top_k, page_size=page)
    q = torch.randn(2, draft, 8, 128, generator=gen).bfloat16().to(DEV)
    mask = torch.tensor([[1, 3], [1, 3]], dtype=torch.int64, device=DEV)
    check_attend(q, k, v, table, n, mask, slots)


def test_attend_many_requests():
    """More requests than a workgroup has threads, many of them empty."""
    gen = torch.Generator().manual_seed(18)
    lens = [(x * 37) % 90 if x % 3 else 0 for x in range(600)]
    k, v, table, n = make_cache(gen, lens, 16, 2, 64, torch.bfloat16)
    q = torch.randn(600, 1, 4, 64, generator=gen).bfloat16().to(DEV)
    check_attend(q, k, v, table, n)


def test_attend_far_offsets():
    """Rows more than 2^32 bytes into the cache."""
    dim, kv, page = 128, 8, 64
    pages = (1 << 32) // (page * kv * dim * 2) + 3
    k = torch.empty(pages, page, kv, dim, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device=DEV)
    gen = torch.Generator().manual_seed(19)
    for x in (k, v):
        x[table[0].long()] = torch.randn(3, page, kv, dim, generator=gen).bfloat16().to(DEV)
    n = torch.tensor([150], dtype=torch.int32, device=DEV)
    q = torch.randn(1, 1, 8, dim, generator=gen).bfloat16().to(DEV)
    out, lse = vts.tree_attention(q, k, v, table, n, return_lse=True)
    near = table.clone()
    order = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)
    small_k, small_v = k[[0, pages - 2, pages - 1]].clone(), v[[0, pages - 2, pages - 1]].clone()
    near[0] = order
    out2, lse2 = vts.tree_attention(q, small_k, small_v, near, n, return_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    check_attend(q, small_k, small_v, near, n)
    w = [torch.zeros(1, kv, 192, device=DEV) for _ in range(2)]
    vts.attention_weight_add(w[0], q, k, table, n, lse)
    vts.attention_weight_add(w[1], q, small_k, near, n, lse)
    assert torch.equal(*w)
    outs = []
    for kk, vv, tt in ((k, v, table), (small_k, small_v, near)):
        ko = torch.zeros(2, page, kv, dim, dtype=k.dtype, device=DEV)
        vo = torch.zeros_like(ko)
        to = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
        vts.evict_cache(w[0], kk, vv, tt, n, 100, ko, vo, to, sinks=2, recent=10)
        outs.append((ko, vo))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_attend_repeats_and_shares_workspaces():
    """The same bits every time, whatever ran in the workspace before."""
    gen = torch.Generator().manual_seed(20)
    a = make_cache(gen, [900, 50, 2000], 16, 2, 128, torch.bfloat16)
    qa = torch.randn(3, 2, 16, 128, generator=gen).bfloat16().to(DEV)
    b = make_cache(gen, [3000], 16, 1, 64, torch.float16)
    qb = torch.randn(1, 5, 20, 64, generator=gen).half().to(DEV)
    probs = torch.softmax(torch.randn(4, 3, 5000, generator=gen), -1).to(DEV)
    toks = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    u = torch.rand(4, 3, generator=gen).to(DEV)
    first = [vts.tree_attention(qa, *a)[0], vts.tree_attention(qb, *b)[0],
             vts.verify_draft(probs, toks, u)[2]]
    for _ in range(5):
        again = [vts.tree_attention(qa, *a)[0], vts.tree_attention(qb, *b)[0],
                 vts.verify_draft(probs, toks, u)[2]]
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_own_workspace():
    gen = torch.Generator().manual_seed(23)
    k, v, table, n = make_cache(gen, [900, 50], 16, 2, 128, torch.bfloat16)
    q = torch.randn(2, 2, 16, 128, generator=gen).bfloat16().to(DEV)
    need = vts.decode.tree_attention_workspace_bytes(2, 2, 16, 2, 128)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    want = vts.tree_attention(q, k, v, table, n)[0]
    assert torch.equal(vts.tree_attention(q, k, v, table, n, workspace=ws)[0], want)
    tickets = ws[:65536].clone()
    assert not tickets.any()  # left as they were
    with pytest.raises(vts.VtsError):
        vts.tree_attention(q, k, v, table, n, workspace=ws[: need - 256])
    with pytest.raises(ValueError, match="workspace"):
        vts.tree_attention(q, k, v, table, n, workspace=ws.cpu())
    probs = torch.softmax(torch.randn(2, 3, 9000, generator=gen), -1).to(DEV)
    toks, u = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.rand(2, 3, generator=gen).to(DEV)
    ws = torch.zeros(vts.decode.verify_draft_workspace_bytes(2, 9000), dtype=torch.uint8, device=DEV)
    want = vts.verify_draft(probs, toks, u)
    assert all(torch.equal(a, b) for a, b in zip(want, vts.verify_draft(probs, toks, u, workspace=ws)))


def test_streams():
    """A stream that is not the current one: its own outputs and workspace."""
    gen = torch.Generator().manual_seed(21)
    k, v, table, n = make_cache(gen, [900, 50], 16, 2, 128, torch.bfloat16)
    q = torch.randn(2, 2, 16, 128, generator=gen).bfloat16().to(DEV)
    want, want_lse = vts.tree_attention(q, k, v, table, n, return_lse=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        out, lse = vts.tree_attention(q, k, v, table, n, return_lse=True, stream=stream)
        w = torch.zeros(2, 2, table.shape[1] * 16, device=DEV)
        torch.cuda.synchronize()
        vts.attention_weight_add(w, q, k, table, n, lse, stream=stream)
        s.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert abs(w.sum().item() - 2 * 2 * 16) < 1e-2


def test_graph_of_a_decode_step():
    """All four calls captured once and replayed with new inputs."""
    gen = torch.Generator().manual_seed(22)
    lens, page, draft, kv, vocab = [400, 90], 16, 3, 2, 5000
    k, v, table, n = make_cache(gen, lens, page, kv, 64, torch.bfloat16, extra_width=3)
    q = torch.randn(2, draft, 8, 64, generator=gen).bfloat16().to(DEV)
    weights = torch.zeros(2, kv, table.shape[1] * page, device=DEV)
    target = torch.softmax(torch.randn(2, draft + 1, vocab, generator=gen), -1).to(DEV)
    drafts = torch.softmax(torch.randn(2, draft, vocab, generator=gen), -1).to(DEV)
    tokens = torch.randint(0, vocab, (2, draft), generator=gen, dtype=torch.int32).to(DEV)
    u = torch.rand(2, draft + 1, generator=gen).to(DEV)
    ko = torch.zeros(2 * 4, page, kv, 64, dtype=k.dtype, device=DEV)
    vo = torch.zeros_like(ko)
    to = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)

    def step():
        out, lse = vts.tree_attention(q, k, v, table, n, return_lse=True)
        path, count, token = vts.verify_draft(target, tokens, u, draft_probs=drafts)
        vts.attention_weight_add(weights, q, k, table, n, lse)
        kept, left, w = vts.evict_cache(weights, k, v, table, n, 60, ko, vo, to, sinks=2, recent=8)
        return out, lse, path, count, token, kept, left, w

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step()
    for i in range(4):
        q.copy_(torch.randn(q.shape, generator=gen).bfloat16())
        u.copy_(torch.rand(u.shape, generator=gen))
        n.copy_(torch.tensor([400 - 50 * i, 90 + i], dtype=torch.int32))
        weights.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in got] + [weights.clone(), ko.clone(), vo.clone()]
        weights.zero_()
        eager = list(step()) + [weights.clone(), ko.clone(), vo.clone()]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, eager))


# ---------------------------------------------------------------- accumulated weight


@pytest.mark.parametrize("i", range(len(CASES)))
def test_weigh(i):
    lens, draft, heads, kv, dim, page, tree, dtype = CASES[i]
    say("weigh", CASES[i])
    gen = torch.Generator().manual_seed(200 + i)
    k, v, table, n = make_cache(gen, lens, page, kv, dim, dtype)
    q = (1.5 * torch.randn(len(lens), draft, heads, dim, generator=gen)).to(dtype).to(DEV)
    mask = random_mask(gen, len(lens), draft)[0] if tree else None
    _, lse = vts.tree_attention(q, k, v, table, n, tree_mask=mask, return_lse=True)
    keep = None
    if i % 2:
        keep = (torch.rand(len(lens), draft, generator=gen) < 0.6).to(DEV)
    width = max(1, max(lens) - (7 if i % 3 == 0 else 0))  # some lists are wider than the weights
    weights = torch.rand(len(lens), kv, width, generator=gen).to(DEV)
    w64, bound = ref.weigh(weights, q, k, table, n, lse, mask, keep)
    got = vts.attention_weight_add(weights, q, k, table, n, lse, tree_mask=mask, row_keep=keep)
    assert got is weights
    worst = ((weights.cpu().double() - w64).abs() / bound).max().item()
    assert worst <= 1, f"{worst:.3g} times the bound"


def test_weigh_leaves_the_rest_alone():
    gen = torch.Generator().manual_seed(30)
    k, v, table, n = make_cache(gen, [50, 0, 70], 16, 2, 64, torch.bfloat16)
    k[table[2, 4].long(), 6:] = math.nan  # past the length
    table[0, 1] = -1
    q = torch.randn(3, 2, 4, 64, generator=gen).bfloat16().to(DEV)
    _, lse = vts.tree_attention(q, k, v, table, n, return_lse=True)
    lse[0, 1] = -math.inf
    big = torch.full((3, 3, 200), 5.0, device=DEV)
    view = big[:, :2, 3:120]
    w64, bound = ref.weigh(view, q, k, table, n, lse)
    vts.attention_weight_add(view, q, k, table, n, lse)
    assert ((view.cpu().double() - w64).abs() <= bound).all()
    assert (view[0, :, 16:32] == 5).all() and (view[1] == 5).all() and (view[2, :, 70:] == 5).all()
    big[:, :2, 3:120] = 5
    assert (big == 5).all()


# ---------------------------------------------------------------- eviction


def check_evict(weights, k, v, table, n, keep, sinks, recent, same_cache=False, out_table=None):
    batch, kv, page = weights.shape[0], k.shape[2], k.shape[1]
    need = -(-keep // page)
    if same_cache:
        ko, vo, base = k, v, k.shape[0] - batch * need
    else:
        ko = torch.full((batch * need + 1, page, kv, k.shape[3]), 9.0, dtype=k.dtype, device=DEV)
        vo, base = torch.full_like(ko, 8.0), 0
    if out_table is None:
        out_table = (base + torch.randperm(batch * need).view(batch, need)).int().to(DEV)
    k0, v0 = k.clone(), v.clone()
    before = (ko.clone(), vo.clone())
    kept, left, w = vts.evict_cache(weights, k, v, table, n, keep, ko, vo, out_table, sinks=sinks,
                                    recent=recent)
    torch.cuda.synchronize()
    want, counts = ref.evict(weights, n.cpu(), table.shape[1] * page, keep, sinks, recent)
    assert left.cpu().tolist() == counts
    fk, fv = k0.reshape(-1, kv, k.shape[3]), v0.reshape(-1, kv, k.shape[3])
    expect_k, expect_v = before
    for b in range(batch):
        for h in range(kv):
            rows = want[b][h]
            assert kept[b, h].cpu().tolist() == rows + [-1] * (keep - len(rows)), (b, h)
            full = torch.zeros(keep, device=DEV)
            at = torch.tensor(rows, dtype=torch.long, device=DEV)
            full[: len(rows)] = weights[b, h, at]
            assert torch.equal(w[b, h].view(torch.int32), full.view(torch.int32))
            if not rows:
                continue
            i = torch.arange(len(rows), device=DEV)
            entry = table[b].long()[at // page]
            there = (entry >= 0) & (entry < k.shape[0])
            src = entry.clamp(0, k.shape[0] - 1) * page + at % page
            dst = out_table[b].long()[i // page]
            fine = (dst >= 0) & (dst < ko.shape[0])
            for old, fx in ((expect_k, fk), (expect_v, fv)):
                vals = torch.where(there[:, None], fx[src, h], 0.0)
                old[dst[fine], (i % page)[fine], h] = vals[fine]
    assert torch.equal(ko.view(torch.int16), expect_k.view(torch.int16))
    assert torch.equal(vo.view(torch.int16), expect_v.view(torch.int16))


@pytest.mark.parametrize("lens,page,kv,dim,keep,sinks,recent", [
    ([0, 1, 99, 100, 101, 350], 16, 2, 64, 100, 4, 20),
    ([300, 40], 24, 3, 128, 64, 0, 0),
    ([300, 64, 65], 64, 1, 64, 64, 10, 54),       # nothing but sinks and recent entries
    ([5000, 1025, 3000], 16, 2, 64, 1024, 1, 7),  # many tiles
    ([16383, 16384, 16385, 30000], 64, 1, 64, 9000, 4, 100),
    ([9, 8, 7], 1, 2, 64, 1, 0, 1),
    ([9, 8, 7], 1, 2, 64, 1, 0, 0),
])
def test_evict(lens, page, kv, dim, keep, sinks, recent):
    say("evict", lens, keep, sinks, recent)
    gen = torch.Generator().manual_seed(40)
    k, v, table, n = make_cache(gen, lens, page, kv, dim, torch.bfloat16)
    u = torch.rand(len(lens), kv, table.shape[1] * page, generator=gen)
    weights = torch.where(u < 0.3, 0.0, (u * 8).round() / 8).to(DEV)  # many ties
    check_evict(weights, k, v, table, n, keep, sinks, recent)
    check_evict(torch.rand(weights.shape, generator=gen).to(DEV), k, v, table, n, keep, sinks, recent)


def test_evict_special_weights():
    gen = torch.Generator().manual_seed(41)
    k, v, table, n = make_cache(gen, [64, 64], 16, 2, 64, torch.float16)
    w = torch.randn(2, 2, 64, generator=gen)
    pool = [math.nan, -math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-45, -1e-45]
    w[0] = torch.tensor(np.random.default_rng(0).choice(pool, (2, 64)).astype(np.float32))
    w[0, 0].view(torch.int32)[::9] = 0x7F800001  # another NaN
    w[0, 1].view(torch.int32)[::9] = -1          # a negative NaN
    w[1, 0] = 0.0
    for keep in (10, 33, 50):
        check_evict(w.to(DEV), k, v, table, n, keep, 3, 5)


def test_evict_bad_pages_and_views():
    gen = torch.Generator().manual_seed(42)
    k, v, table, n = make_cache(gen, [64, 90], 16, 2, 64, torch.float16, order="heads_first")
    table[0, 1] = -1
    table[1, 2] = 10 ** 6
    out_table = torch.tensor([[0, -1, 1], [2, 7, 3]], dtype=torch.int32, device=DEV)
    weights = torch.rand(2, 3, 100, generator=gen).to(DEV)[:, :2, :95]  # narrower than the table
    check_evict(weights, k, v, table, n, 40, 2, 4, out_table=out_table)


def test_evict_into_the_same_cache():
    gen = torch.Generator().manual_seed(43)
    k, v, table, n = make_cache(gen, [90, 70], 16, 2, 64, torch.bfloat16)
    more = torch.zeros(8, 16, 2, 64, dtype=k.dtype, device=DEV)
    k, v = torch.cat([k, more]), torch.cat([v, more])
    weights = torch.rand(2, 2, 96, generator=gen).to(DEV)
    check_evict(weights, k, v, table, n, 50, 1, 9, same_cache=True)


# ---------------------------------------------------------------- verification


def check_verify(target, tokens, u, drafts=None, parents=None, **kw):
    dev = [None if x is None else x.to(DEV) for x in (target, tokens, u, drafts, parents)]
    path, count, token = vts.verify_draft(dev[0], dev[1], dev[2], draft_probs=dev[3],
                                          parents=dev[4], **kw)
    torch.cuda.synchronize()
    paths, nexts = ref.verify(target, tokens, u, drafts, parents)
    n = tokens.shape[1]
    assert count.cpu().tolist() == [len(p) for p in paths]
    assert path.cpu().tolist() == [p + [-1] * (n - len(p)) for p in paths]
    assert token.cpu().tolist() == nexts
    return paths, nexts


def random_tree(gen, batch, draft, branch):
    p = torch.full((batch, draft), -1)
    for b in range(batch):
        for t in range(1, draft):
            p[b, t] = t // branch - 1 if branch else torch.randint(-1, t, (1,), generator=gen)
    return p.int()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("batch,draft,vocab,branch,drawn", [
    (5, 3, 1000, 1, True), (5, 3, 1000, 1, False), (3, 1, 1, 1, True), (4, 2, 5, 1, False),
    (8, 12, 20011, 3, True), (8, 12, 20011, 3, False), (2, 64, 300, 0, True),
    (2, 64, 300, 0, False), (1, 2, 131072, 1, True), (64, 4, 4097, 2, True),
])
def test_verify(dtype, batch, draft, vocab, branch, drawn):
    say("verify", dtype, batch, draft, vocab, branch, drawn)
    gen = torch.Generator().manual_seed(vocab + draft)
    base = 2 * torch.randn(batch, draft + 1, vocab, generator=gen)
    target = torch.softmax(base, -1).to(dtype)
    near = torch.softmax(base[:, :draft] + 0.8 * torch.randn(batch, draft, vocab, generator=gen), -1)
    parents = None if branch == 1 else random_tree(gen, batch, draft, branch)
    rows = torch.arange(draft).expand(batch, -1) if parents is None else parents.long() + 1
    dist = near.gather(1, rows[..., None].expand(-1, -1, vocab))
    tokens = torch.multinomial(dist.reshape(-1, vocab), 1, generator=gen).view(batch, draft).int()
    for _ in range(3):
        u = torch.rand(batch, draft + 1, generator=gen)
        check_verify(target, tokens, u, near.to(dtype) if drawn else None, parents)


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_ends(drawn):
    """Numbers at the ends of [0, 1), tokens of no probability, all accepted, none."""
    gen = torch.Generator().manual_seed(50)
    vocab = 3001
    target = torch.softmax(torch.randn(4, 4, vocab, generator=gen), -1)
    drafts = torch.softmax(torch.randn(4, 3, vocab, generator=gen), -1) if drawn else None
    tokens = torch.randint(0, vocab, (4, 3), generator=gen).int()
    target[0, 0, tokens[0, 0]] = 0
    target[1, :, :7] = 0
    target[2, :, -9:] = 0
    one = 1 - 2.0 ** -24
    for last in (0.0, one):
        for u in (0.0, one):
            x = torch.full((4, 4), u)
            x[:, 3] = last
            check_verify(target, tokens, x, drafts)


def test_verify_no_mass_left():
    """Residuals without mass fall back to the target, targets without mass give -1."""
    target = torch.zeros(4, 3, 100)
    target[:, :, 10] = 0.25  # less than the draft everywhere
    target[1] = 0
    target[2, :, 11] = math.nan
    target[3, :, 12] = -1
    drafts = torch.zeros(4, 2, 100)
    drafts[:, :, 10] = 1.0
    tokens = torch.full((4, 2), 10, dtype=torch.int32)
    u = torch.full((4, 3), 0.9)
    paths, nexts = check_verify(target, tokens, u, drafts)
    assert nexts == [10, -1, 10, 10] and paths == [[]] * 4
    check_verify(target, tokens, u, None)


def test_verify_bad_nodes():
    """Tokens outside the vocabulary and parents that are no earlier node."""
    gen = torch.Generator().manual_seed(52)
    target = torch.softmax(torch.randn(2, 7, 50, generator=gen), -1)
    drafts = torch.softmax(torch.randn(2, 6, 50, generator=gen), -1)
    tokens = torch.tensor([[-1, 50, 3, 2 ** 31 - 1, 4, 5], [1, 2, 3, 4, 5, 6]], dtype=torch.int32)
    parents = torch.tensor([[-1, -1, -1, 2, 2, 4], [-2, 5, 2 ** 31 - 1, -2 ** 31, -1, 4]],
                           dtype=torch.int32)
    for u in (0.0, 0.3, 0.99):
        x = torch.full((2, 7), u)
        check_verify(target, tokens, x, drafts, parents)
        check_verify(target, tokens, x, None, parents)


def test_verify_same_token_twice():
    gen = torch.Generator().manual_seed(53)
    target = torch.softmax(torch.randn(16, 5, 40, generator=gen), -1)
    drafts = torch.softmax(torch.randn(16, 4, 40, generator=gen), -1)
    tokens = torch.tensor([[3, 3, 5, 3]] * 16, dtype=torch.int32)
    parents = torch.full((16, 4), -1, dtype=torch.int32)
    u = torch.rand(16, 5, generator=gen)
    check_verify(target, tokens, u, drafts, parents)
    check_verify(target, tokens, u, None, parents)


def test_verify_strides():
    gen = torch.Generator().manual_seed(54)
    target = torch.softmax(torch.randn(3, 3, 777, generator=gen), -1).to(DEV)
    drafts = torch.softmax(torch.randn(3, 2, 777, generator=gen), -1).to(DEV)
    tokens = torch.randint(0, 777, (3, 2), generator=gen).int().to(DEV)
    u = torch.rand(3, 3, generator=gen).to(DEV)
    want = vts.verify_draft(target, tokens, u, draft_probs=drafts)
    wide = torch.full((3, 4, 900), 7.0, device=DEV)
    wide[:, :3, 5:782] = target
    shared = torch.full((2, 3, 801), 7.0, device=DEV)
    shared[:, :, 1:778] = drafts.transpose(0, 1)
    got = vts.verify_draft(wide[:, :3, 5:782], tokens, u, draft_probs=shared[:, :, 1:778].transpose(0, 1))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_gives_the_targets_distribution(drawn):
    """The first token of the outcome is distributed as the target's first row."""
    gen = torch.Generator().manual_seed(55)
    batch, vocab = 40000, 6
    p = torch.tensor([0.3, 0.25, 0.2, 0.15, 0.1, 0.0])
    q = torch.tensor([0.1, 0.1, 0.4, 0.1, 0.2, 0.1])
    target = p.expand(batch, 4, vocab).contiguous().to(DEV)
    drafts = q.expand(batch, 3, vocab).contiguous().to(DEV)
    parents = torch.tensor([-1, -1, -1], dtype=torch.int32).expand(batch, -1).contiguous().to(DEV)
    tokens = torch.multinomial(q.expand(batch * 3, vocab), 1, generator=gen).view(batch, 3).int()
    u = torch.rand(batch, 4, generator=gen).to(DEV)
    path, count, token = vts.verify_draft(target, tokens.to(DEV), u,
                                          draft_probs=drafts if drawn else None, parents=parents)
    first = torch.where(count.cpu() > 0, tokens.gather(1, path.cpu()[:, :1].clamp(min=0).long())[:, 0],
                        token.cpu())
    share = torch.bincount(first.long(), minlength=vocab).double() / batch
    # five standard deviations of a share
    assert ((share - p.double()).abs() <= 5 * (p.double() * (1 - p.double()) / batch).sqrt()).all()
