"""tree_attention over microscaled caches against plain 64-bit forms of the values they stand for
(tests/decode_ref.py), under the bounds that hold for 16-bit caches: every form of workgroup, lengths
from zero on, masks, layouts, slot lists, pages that are not there, blocks of NaN, graphs, streams."""
import math

import pytest
import torch

import varlen_top_select_amd as vts
from tests import cache_ref, decode_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16


def say(*a):
    print(*a, flush=True)


def laid_out(t, order):
    if order == "heads_first":
        return t.permute(0, 2, 1, 3).contiguous().to(DEV).permute(0, 2, 1, 3)
    if order == "padded":
        n, page, kv, w = t.shape
        wide = torch.zeros(n, page, kv + 1, w + (16 if w >= 32 else w), dtype=t.dtype, device=DEV)
        wide[:, :, :kv, :w] = t.to(DEV)
        return wide[:, :, :kv, :w]
    return t.to(DEV)


def make_cache(gen, lens, page, kv, dim, bits, order=None, extra_width=1):
    """(caches, scales, their values in float64, page table, lengths)"""
    used = [-(-max(x, 0) // page) for x in lens]
    width = max(used + [1]) + extra_width
    pool = sum(used) + 2
    perm = torch.randperm(pool, generator=gen)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(used):
        table[b, :m] = perm[at:at + m].int()
        at += m
    caches, scales, deep = [], [], []
    for _ in "kv":
        codes = torch.randint(0, 16 if bits == 4 else 128, (pool, page, kv, dim), generator=gen)
        if bits == 8:  # magnitudes up to 240, either sign
            codes = codes.clamp(max=0x77) | torch.randint(0, 2, codes.shape, generator=gen) << 7
        # blocks of very different sizes, the largest about 1 to 8
        high = 127 - (2 if bits == 4 else 7)
        scale = torch.randint(high - 4, high + 2, (pool, page, kv, dim // 32), generator=gen)
        deep.append(cache_ref.values(codes, scale, bits))
        caches.append(laid_out(cache_ref.pack(codes, bits), order))
        scales.append(laid_out(scale.to(torch.uint8), order))
    return caches, scales, deep, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def random_mask(gen, batch, draft):
    parents = torch.stack([torch.cat([torch.tensor([-1])] + [
        torch.randint(-1, t, (1,), generator=gen) for t in range(1, draft)]) for _ in range(batch)])
    return vts.tree_mask_from_parents(parents.int()).to(DEV)


def check(q, caches, scales, deep, table, lens, mask=None, slots=None, scale=None, **kw):
    out, lse = vts.tree_attention(q, *caches, table, lens, tree_mask=mask, slots=slots, scale=scale,
                                  return_lse=True, k_scales=scales[0], v_scales=scales[1], **kw)
    torch.cuda.synchronize()
    o64, l64, mag, reach = ref.attend(q, *deep, table, lens, mask, slots, scale)
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
    # lengths, draft, heads, kv, dim, page, tree, dtype, layout
    ([1], 1, 1, 1, 64, 16, False, BF16, None),
    ([0, 1, 2, 31, 32, 33], 1, 8, 2, 128, 16, False, BF16, None),
    ([0, 1, 2, 3, 4, 5, 127, 128, 129, 130], 3, 6, 3, 64, 1, False, F16, "padded"),
    ([5, 300, 7, 1000], 5, 14, 2, 64, 24, True, F16, None),
    ([64, 65, 63, 700], 4, 32, 8, 128, 64, True, BF16, "heads_first"),
    ([200, 90], 7, 24, 2, 128, 7, True, BF16, None),      # 84 rows: a wide workgroup, not full
    ([150, 64, 40], 64, 4, 2, 64, 16, True, F16, None),   # 64 drafted tokens, a length below
    ([2500], 2, 16, 1, 128, 128, False, F16, None),       # one list over many workgroups
    ([777, 1, 300], 1, 40, 1, 128, 32, False, BF16, "padded"),
    # four heads or a multiple and many lists: a head to a wave
    ([(x * 61) % 300 for x in range(16)] + [2000] * 16, 1, 16, 4, 64, 16, False, BF16, None),
    ([100] * 31 + [3000], 2, 16, 4, 128, 32, True, F16, "heads_first"),
    ([90, 0, 1, 400] * 8, 5, 32, 4, 128, 24, True, BF16, None),  # 40 rows each: wide
    ([33, 65, 200, 0] * 8, 4, 32, 4, 128, 16, True, BF16, None),  # 32 rows, a head to a wave
    ([33, 65, 200, 0] * 8, 4, 32, 4, 64, 16, True, F16, None),
    ([9000], 1, 2, 1, 64, 64, False, BF16, None),  # blocks of parts
    # wide: 64, 128 rows and more to a KV head, lists that end anywhere
    ([1, 0, 63, 64, 65, 129, 700], 16, 8, 2, 128, 16, True, BF16, None),
    ([1500, 17], 20, 12, 2, 64, 24, True, F16, "heads_first"),
    ([700, 129, 64], 40, 8, 2, 128, 32, True, F16, "padded"),
    ([600, 70], 64, 10, 2, 64, 64, False, BF16, None),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_paged(i, bits):
    lens, draft, heads, kv, dim, page, tree, dtype, order = CASES[i]
    say("attend", bits, CASES[i])
    gen = torch.Generator().manual_seed(500 + i)
    caches, scales, deep, table, n = make_cache(gen, lens, page, kv, dim, bits, order)
    q = (0.7 * torch.randn(len(lens), draft, heads, dim, generator=gen)).to(dtype).to(DEV)
    mask = random_mask(gen, len(lens), draft) if tree else None
    check(q, caches, scales, deep, table, n, mask)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("heads,kv,dim,top_k,tree,draft", [
    (8, 2, 128, 70, True, 3), (16, 1, 64, 33, False, 2), (64, 2, 128, 100, True, 2),
    (130, 1, 64, 257, True, 1), (7, 7, 128, 1, False, 1)])
def test_slots(bits, heads, kv, dim, top_k, tree, draft):
    gen = torch.Generator().manual_seed(60)
    caches, scales, deep, table, n = make_cache(gen, [300, 41, 0], 16, kv, dim, bits)
    total = caches[0].shape[0] * 16
    slots = torch.randint(0, total, (3, draft, top_k), generator=gen).int()
    slots[torch.rand(slots.shape, generator=gen) < 0.2] = -1
    slots[torch.rand(slots.shape, generator=gen) < 0.05] = total
    slots[1, 0] = -1  # a row that lists nothing
    q = (0.7 * torch.randn(3, draft, heads, dim, generator=gen)).bfloat16().to(DEV)
    mask = random_mask(gen, 3, draft) if tree else None
    check(q, caches, scales, deep, table, n, mask, slots.to(DEV))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("heads,kv,dim,top_k,tree,draft,batch,dtype", [
    (16, 4, 128, 70, True, 3, 12, BF16), (16, 4, 64, 33, False, 2, 16, F16), (64, 4, 128, 100, True, 2, 16, F16),
    (96, 4, 128, 40, True, 1, 32, BF16), (8, 8, 64, 300, True, 2, 8, BF16), (128, 4, 128, 65, True, 1, 32, BF16)])
def test_many_slot_lists(bits, heads, kv, dim, top_k, tree, draft, batch, dtype):
    """A KV head to each wave, 16 and 32 rows, lists shared by several workgroups, and more rows."""
    gen = torch.Generator().manual_seed(68)
    lens = [(61 * x) % 190 for x in range(batch)]
    caches, scales, deep, table, n = make_cache(gen, lens, 16, kv, dim, bits)
    total = caches[0].shape[0] * 16
    slots = torch.randint(0, total, (batch, draft, top_k), generator=gen).int()
    slots[torch.rand(slots.shape, generator=gen) < 0.2] = -1
    slots[1, 0] = -1
    q = (0.7 * torch.randn(batch, draft, heads, dim, generator=gen)).to(dtype).to(DEV)
    mask = random_mask(gen, batch, draft) if tree else None
    check(q, caches, scales, deep, table, n, mask, slots.to(DEV))


@pytest.mark.parametrize("bits", [4, 8])
def test_pages_that_are_not_there(bits):
    gen = torch.Generator().manual_seed(61)
    caches, scales, deep, table, n = make_cache(gen, [200, 100, 50], 16, 2, 128, bits)
    table[0, 3] = -1
    table[0, 7] = caches[0].shape[0]
    table[1] = 2 ** 31 - 1
    table[2, :2] = -2 ** 31
    q = torch.randn(3, 2, 8, 128, generator=gen).bfloat16().to(DEV)
    check(q, caches, scales, deep, table, n)
    lens = torch.tensor([2 ** 31 - 1, -5, 50], dtype=torch.int32, device=DEV)  # clamped
    check(q, caches, scales, deep, table, lens)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("draft,heads,kv", [(3, 8, 2), (4, 16, 4), (16, 8, 2), (40, 8, 2), (6, 16, 4)])
def test_nan_where_it_is_not_seen(bits, draft, heads, kv):
    """Blocks of NaN behind the length, on pages of nobody, and at drafted tokens that some rows do
    not see: those rows get what they would get without them, and the rows that see them NaN."""
    gen = torch.Generator().manual_seed(62)
    lens = [70 + draft, 33, 130] * (16 if kv == 4 else 1)  # (a head to a wave with many lists)
    caches, scales, deep, table, n = make_cache(gen, lens, 16, kv, 128, bits)
    q = torch.randn(len(lens), draft, heads, 128, generator=gen).bfloat16().to(DEV)
    lens = torch.tensor(lens)
    clean, clean_lse = vts.tree_attention(q, *caches, table, n, k_scales=scales[0], v_scales=scales[1],
                                          return_lse=True)
    bad = 1  # drafted token of request 0: rows 1.. of the chain see it
    pos = int(lens[0]) - draft + bad
    page, at = int(table[0, pos // 16]), pos % 16
    used = torch.zeros(caches[0].shape[0], 16, dtype=torch.bool)
    for b in range(len(lens)):
        for j in range(int(lens[b])):
            used[int(table[b, j // 16]), j % 16] = True
    for which, s in enumerate(scales):
        s[~used.to(DEV)] = 255
        if which == 1:
            s[page, at, :, 2] = 255  # elements 64..95 of V
    got, lse = vts.tree_attention(q, *caches, table, n, k_scales=scales[0], v_scales=scales[1],
                                  return_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(lse, clean_lse)
    seen = torch.zeros(got.shape, dtype=torch.bool)
    seen[0, bad:, :, 64:96] = True
    got, clean = got.cpu(), clean.cpu()
    assert got[seen].isnan().all()
    assert torch.equal(got[~seen], clean[~seen])


def test_infinite_values_of_fp16():
    """Numbers past fp16's range are infinities to fp16 queries; rows that do not see them do not
    get them."""
    gen = torch.Generator().manual_seed(63)
    caches, scales, deep, table, n = make_cache(gen, [40], 16, 1, 64, 8)
    q = torch.randn(1, 4, 4, 64, generator=gen).half().to(DEV)
    clean, _ = vts.tree_attention(q, *caches, table, n, k_scales=scales[0], v_scales=scales[1])
    pos = 38  # drafted token 2
    page, at = int(table[0, pos // 16]), pos % 16
    caches[1][page, at, 0, :32] = 0x70  # 128
    scales[1][page, at, 0, 0] = 127 + 10  # * 2^10
    got, _ = vts.tree_attention(q, *caches, table, n, k_scales=scales[0], v_scales=scales[1])
    assert torch.equal(got[0, :2], clean[0, :2])
    assert (got[0, 2:, :, :32] == math.inf).all()
    assert torch.equal(got[0, 2:, :, 32:].isfinite(), torch.ones_like(got[0, 2:, :, 32:], dtype=torch.bool))


@pytest.mark.parametrize("bits", [4, 8])
def test_strides_streams_workspace_and_scale(bits):
    gen = torch.Generator().manual_seed(64)
    caches, scales, deep, table, n = make_cache(gen, [70, 200, 33], 16, 3, 128, bits, "padded")
    # q as [batch, heads, draft, dim] seen the other way round, the table as a slice
    q = (0.7 * torch.randn(3, 6, 2, 128, generator=gen)).bfloat16().to(DEV).transpose(1, 2)
    wide = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    wide[:, 2:2 + table.shape[1]] = table
    view = wide[:, 2:2 + table.shape[1]]
    for s in (None, 0.3, -0.2, 0.0):
        want, _ = check(q, caches, scales, deep, view, n, scale=s)
    want, lse = check(q, caches, scales, deep, view, n)
    ws = torch.zeros(vts.decode.tree_attention_workspace_bytes(3, 2, 6, 3, 128, 0, True), dtype=torch.uint8,
                     device=DEV)
    out = torch.full_like(want, 3.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, _ = vts.tree_attention(q, *caches, view, n, k_scales=scales[0], v_scales=scales[1], out=out,
                                workspace=ws, stream=side)
    side.synchronize()
    assert got is out and torch.equal(got, want) and not ws[:65536].any()
    with pytest.raises(vts.VtsError):
        vts.tree_attention(q, *caches, view, n, k_scales=scales[0], v_scales=scales[1], workspace=ws[:-256])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("batch,draft,heads,kv", [(3, 2, 8, 2), (40, 1, 16, 4), (2, 16, 16, 2)])
def test_graph(bits, batch, draft, heads, kv):
    gen = torch.Generator().manual_seed(65)
    lens = [500 + 37 * b % 200 for b in range(batch)]
    caches, scales, deep, table, n = make_cache(gen, lens, 16, kv, 128, bits)
    q = torch.randn(batch, draft, heads, 128, generator=gen).bfloat16().to(DEV)
    kw = dict(k_scales=scales[0], v_scales=scales[1], return_lse=True)
    ws = torch.zeros(vts.decode.tree_attention_workspace_bytes(batch, draft, heads, kv, 128, 0, True),
                     dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = vts.tree_attention(q, *caches, table, n, workspace=ws, **kw)
    for turn in range(4):
        n.sub_(turn * 13)
        q.mul_(1.1)
        out.zero_()
        want, want_lse = vts.tree_attention(q, *caches, table, n, **kw)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse), turn


@pytest.mark.parametrize("bits", [4, 8])
def test_places_past_4_gib(bits):
    """Rows beyond 2^32 bytes of a cache, and scales beyond 2^28 rows of them."""
    row = 128 * bits // 8
    pages = (5 << 30) // (64 * 8 * row)
    kc, vc = (torch.zeros(pages, 64, 8, row, dtype=torch.uint8, device=DEV) for _ in "kv")
    ks, vs = (torch.zeros(pages, 64, 8, 4, dtype=torch.uint8, device=DEV) for _ in "kv")
    gen = torch.Generator().manual_seed(66)
    caches, scales, deep, table, n = make_cache(gen, [130], 64, 8, 128, bits)
    far = torch.tensor([[pages - 1, pages * 13 // 16, pages - 9, -1]], dtype=torch.int32, device=DEV)
    for i in range(3):
        for big, small in zip((kc, vc, ks, vs), (*caches, *scales)):
            big[int(far[0, i])] = small[int(table[0, i])]
    for heads, draft in ((8, 1), (64, 4), (64, 16)):
        q = (0.5 * torch.randn(1, draft, heads, 128, generator=gen)).bfloat16().to(DEV)
        want = vts.tree_attention(q, *caches, table, n, k_scales=scales[0], v_scales=scales[1])[0]
        got = vts.tree_attention(q, kc, vc, far, n, k_scales=ks, v_scales=vs)[0]
        assert torch.equal(got, want)


def test_a_request_from_its_prompt_on():
    """A prompt in two chunks into a 4-bit cache, then decode steps: the way the operators are used
    together, against 64-bit forms of the same."""
    gen = torch.Generator().manual_seed(67)
    heads, kv, dim, page, bits = 8, 2, 128, 16, 4
    lens, chunk = [90, 41], [50, 41]
    total = sum(lens)
    table = torch.randperm(16, generator=gen)[:14].view(2, 7).int().to(DEV)
    kc, vc = (torch.zeros(16, page, kv, dim // 2, dtype=torch.uint8, device=DEV) for _ in "kv")
    ks, vs = (torch.zeros(16, page, kv, dim // 32, dtype=torch.uint8, device=DEV) for _ in "kv")
    cache = dict(k_scales=ks, v_scales=vs)
    rotary = vts.rotary_table(256, dim, device=DEV)
    w = [(1 + 0.2 * torch.randn(dim, generator=gen)).bfloat16().to(DEV) for _ in "qk"]
    x = [torch.randn(n + 3, heads + 2 * kv, dim, generator=gen).bfloat16() for n in lens]

    def step(spans):
        """write_cache of positions [a, b) of each request; queries, keys."""
        rows = torch.cat([x[b][a:e] for b, (a, e) in enumerate(spans)]).to(DEV)
        most = max(e - a for a, e in spans)
        pos = torch.stack([torch.arange(a, a + most) for a, _ in spans]).to(DEV)
        real = torch.stack([torch.arange(most) < e - a for a, e in spans]).to(DEV)
        slots = vts.page_slots(table, page, pos)[real]
        return (*vts.write_cache(rows[:, :heads], rows[:, heads:heads + kv], rows[:, heads + kv:], slots, kc, vc,
                                 positions=pos[real].int(), rotary=rotary, q_norm=w[0], k_norm=w[1],
                                 return_k=True, **cache), rows[:, heads + kv:])

    def cu(n):
        return torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32, device=DEV)

    # the first part of each prompt, attended as it is
    q1, k1, v1 = step([(0, n) for n in chunk])
    out1, _ = vts.prompt_attention(q1, k1, v1, cu(chunk))
    o64, l64, mag, reach = cache_ref.prompt(q1, k1, v1, cu(chunk), cu(chunk))
    ob, _ = ref.attend_bounds(o64, mag, reach, max(chunk), dim, BF16)
    assert ((out1.cpu().double() - o64).abs() <= ob).all()
    # the rest of the first prompt behind what is cached
    rest = [n - c for n, c in zip(lens, chunk)]
    q2, k2, v2 = step([(c, n) for c, n in zip(chunk, lens)])
    pos = torch.arange(max(lens), device=DEV).expand(2, -1)
    every = vts.page_slots(table, page, pos)[pos < torch.tensor(lens, device=DEV)[:, None]]
    kk, vv = vts.read_cache(kc, vc, every, dtype=BF16, **cache)
    out2, _ = vts.prompt_attention(q2, kk, vv, cu(rest), cu_seqlens_k=cu(lens))
    o64, l64, mag, reach = cache_ref.prompt(q2, kk, vv, cu(rest), cu(lens))
    ob, _ = ref.attend_bounds(o64, mag, reach, max(lens), dim, BF16)
    assert ((out2.cpu().double() - o64).abs() <= ob).all()
    # what was read back is the quantised form of what was written
    assert torch.equal(vv[:chunk[0]].cpu().double(), ref_rows(v1[:chunk[0]], bits))
    # a decode step of three drafted tokens each
    q3, _, _ = step([(n, n + 3) for n in lens])
    n3 = torch.tensor([n + 3 for n in lens], dtype=torch.int32, device=DEV)
    deep = []
    for c, s in ((kc, ks), (vc, vs)):
        deep.append(cache_ref.values(cache_ref.unpack(c.cpu(), bits), s.cpu(), bits))
    check(q3.view(2, 3, heads, dim), (kc, vc), (ks, vs), deep, table, n3)


def ref_rows(x, bits):
    return cache_ref.values(*cache_ref.quantise(x.cpu().double(), bits), bits)
