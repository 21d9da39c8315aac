"""write_cache and read_cache against plain 64-bit forms (tests/cache_ref.py): head norms,
positions, 16-, 8- and 4-bit caches of any layout, padding, values at the formats' borders,
what is not finite, streams, graphs, caches past 2^32 bytes."""
import math

import pytest
import torch

import varlen_top_select_amd as vts
from tests import cache_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16


def say(*a):
    print(*a, flush=True)


def memory(gen, pages, page, kv, width, dtype, order=None):
    """A cache tensor of random bytes or values: what must not change is seen if it does."""
    shape = (pages, page, kv, width)
    if order == "heads_first":
        shape = (pages, kv, page, width)
    if order == "padded":
        step = 8 if dtype != torch.uint8 else 16 if width >= 32 else width
        shape = (pages, page, kv + 1, width + step)
    if dtype == torch.uint8:
        t = torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8).to(DEV)
    else:
        t = torch.randn(shape, generator=gen).to(dtype).to(DEV)
    if order == "heads_first":
        t = t.transpose(1, 2)
    return t[:, :, :kv, :width] if order == "padded" else t


def make_cache(gen, pages, page, kv, dim, bits, dtype, order=None):
    if bits == 16:
        return [memory(gen, pages, page, kv, dim, dtype, order) for _ in "kv"], [None, None]
    return ([memory(gen, pages, page, kv, dim * bits // 8, torch.uint8, order) for _ in "kv"],
            [memory(gen, pages, page, kv, dim // 32, torch.uint8, order) for _ in "kv"])


def at_slots(t, slots):
    page = t.shape[1]
    slots = slots.to(t.device).long()
    return t[slots // page, slots % page].cpu()


CASES = [
    # tokens, heads, kv, dim, rot, interleaved, norm, bits, page, order, dtype
    (1, 32, 8, 128, 128, False, True, 4, 64, None, BF16),
    (1, 1, 1, 64, 0, False, False, 8, 1, None, F16),
    (5, 14, 2, 64, 32, True, True, 4, 24, "heads_first", F16),
    (130, 3, 3, 128, 64, False, True, 8, 16, "padded", BF16),
    (77, 8, 1, 128, 128, True, False, 16, 16, "padded", BF16),
    (64, 21, 3, 64, 64, False, True, 16, 7, "heads_first", F16),
    (33, 16, 16, 128, 16, False, False, 4, 128, "padded", F16),
    (700, 4, 4, 64, 48, True, True, 8, 64, "heads_first", BF16),
    (2, 64, 8, 128, 96, False, True, 8, 32, None, F16),
    (5000, 2, 1, 128, 128, False, True, 4, 64, None, BF16),
    (300, 12, 12, 64, 16, True, True, 4, 16, None, BF16),
    (9, 6, 3, 128, 0, False, True, 4, 16, None, BF16),   # norms alone
    (9, 5, 2, 64, 0, False, True, 16, 16, None, F16),
]


def make_tokens(gen, tokens, heads, kv, dim, dtype, scale=2.0):
    """Views of one projection's output."""
    x = (scale * torch.randn(tokens, heads + 2 * kv, dim, generator=gen)).to(dtype).to(DEV)
    return x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_write_and_read(i):
    tokens, heads, kv, dim, rot, inter, norm, bits, page, order, dtype = CASES[i]
    say("write", CASES[i])
    gen = torch.Generator().manual_seed(300 + i)
    q, k, v = make_tokens(gen, tokens, heads, kv, dim, dtype)
    pages = -(-tokens // page) + 3
    (kc, vc), (ks, vs) = make_cache(gen, pages, page, kv, dim, bits, dtype, order)
    slots = torch.randperm(pages * page, generator=gen)[:tokens].int()
    # padding: no slot, or none that exists
    gone = torch.rand(tokens, generator=gen) < (0.2 if tokens > 4 else 0)
    slots[gone] = torch.tensor([-1, pages * page, 2 ** 31 - 1, -2 ** 31])[
        torch.randint(0, 4, (int(gone.sum()),), generator=gen)].int()
    table = positions = None
    if rot:
        table = vts.rotary_table(5000, rot, device=DEV)
        positions = torch.randint(0, 5000, (tokens,), generator=gen).int()
        if tokens > 4:
            positions[torch.randperm(tokens, generator=gen)[:2]] = torch.tensor([-1, 5000]).int()
    qn = kn = None
    if norm:
        qn, kn = ((1 + 0.3 * torch.randn(dim, generator=gen)).to(dtype if i % 2 else torch.float32).to(DEV)
                  for _ in "qk")
    before = [t.clone() for t in (kc, vc, ks, vs) if t is not None]
    want = dict(k_scales=ks, v_scales=vs)
    got_q, got_k = vts.write_cache(
        q, k, v, slots.to(DEV), kc, vc, positions=None if positions is None else positions.to(DEV),
        rotary=table, interleaved=inter, q_norm=qn, k_norm=kn, eps=1e-5, return_k=True, **want)
    torch.cuda.synchronize()
    q64, qm = ref.ready(q, qn, 1e-5, table, positions, inter)
    k64, km = ref.ready(k, kn, 1e-5, table, positions, inter)
    for name, got, y, m in (("q", got_q, q64, qm), ("k", got_k, k64, km)):
        worst = ((got.cpu().double() - y).abs() / ref.ready_bound(y, m, dim, dtype)).max().item()
        assert worst <= 1, f"{name}: {worst:.3g} times its bound"
    live = ~gone
    if rot:
        live &= (positions >= 0) & (positions < 5000)
    used = slots[live]
    v64 = v.cpu().double()
    if bits == 16:
        assert torch.equal(at_slots(kc, used), got_k.cpu()[live])
        assert torch.equal(at_slots(vc, used).view(torch.int16), v.cpu()[live].contiguous().view(torch.int16))
    else:
        for c, s, x in ((kc, ks, k64), (vc, vs, v64)):
            codes, scale = ref.quantise(x[live], bits)
            assert torch.equal(at_slots(s, used).long(), scale)
            assert torch.equal(at_slots(c, used), ref.pack(codes, bits))
    # nothing else has changed
    flat = torch.ones(pages * page, dtype=torch.bool)
    flat[used.long()] = False
    rest = torch.nonzero(flat)[:, 0]
    for t, b in zip([t for t in (kc, vc, ks, vs) if t is not None], before):
        assert torch.equal(at_slots(t, rest), at_slots(b, rest))
    # and what is read back is what the bytes stand for
    rk, rv = vts.read_cache(kc, vc, slots.to(DEV), dtype=dtype, **want)
    torch.cuda.synchronize()
    inside = (slots >= 0) & (slots < pages * page)
    for got, c, s in ((rk, kc, ks), (rv, vc, vs)):
        assert (got.cpu()[~inside] == 0).all()
        x = at_slots(c, slots[inside])
        if bits != 16:
            x = ref.values(ref.unpack(x, bits), at_slots(s, slots[inside]), bits).to(dtype)
        assert torch.equal(got.cpu()[inside].nan_to_num(7.0, 1e30, -1e30), x.nan_to_num(7.0, 1e30, -1e30))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_borders(bits, dtype):
    """Every border of two numbers, one step of dtype to either side of it, at every scale that
    dtype reaches, with the largest magnitude at the format's and past it."""
    grid = ref.numbers(bits)
    tops = [grid[-1], 2 * grid[-1] - grid[-2], (3 * grid[-1] - grid[-2]) / 2, grid[-1] * 1.05, grid[-1] / 2 * 1.3]
    mids = torch.cat([grid, (grid[1:] + grid[:-1]) / 2])
    rows = []
    for top in tops:
        x = mids.to(dtype)
        x = torch.cat([x, torch.nextafter(x, torch.full_like(x, 1e4 if dtype == F16 else 1e9)),
                       torch.nextafter(x, torch.full_like(x, 0))]).double()
        x = torch.where(x > top, top, x)
        x = torch.nn.functional.pad(x, (0, -len(x) % 31))
        x = x.view(-1, 31)
        x = x * torch.where(torch.arange(31) % 3 == 1, -1.0, 1.0)
        x = torch.cat([x, torch.full((len(x), 1), float(top), dtype=torch.float64)], 1)
        for e in (0, -3, 5, 7) if dtype == F16 else (0, -30, 60, -100, 110):
            rows.append(x * 2.0 ** e)
    x = torch.cat(rows).to(dtype)
    x = torch.nn.functional.pad(x, (0, 0, 0, -len(x) % 4)).view(-1, 1, 128)
    n = len(x)
    caches = [torch.zeros(n, 1, 1, 16 * bits, dtype=torch.uint8, device=DEV) for _ in "kv"]
    scales = [torch.zeros(n, 1, 1, 4, dtype=torch.uint8, device=DEV) for _ in "kv"]
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    y = x.to(DEV)
    vts.write_cache(y, y, y, slots, *caches, k_scales=scales[0], v_scales=scales[1])
    codes, scale = ref.quantise(x.double(), bits)
    for c, s in zip(caches, scales):
        assert torch.equal(s.cpu().view(n, 1, 4).long(), scale)
        assert torch.equal(c.cpu().view(n, 1, -1), ref.pack(codes, bits))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_extremes(bits, dtype):
    """The type's largest and smallest values, zeros, and blocks that are not finite."""
    f = torch.finfo(dtype)
    low = torch.tensor([1], dtype=torch.int16).view(dtype).item()  # the least subnormal
    x = torch.zeros(12, 1, 64, dtype=dtype)
    x[0] = f.max
    x[1, :, ::2] = -f.max
    x[2] = low
    x[3, :, 5] = f.tiny
    x[4, :, 3] = math.inf
    x[5, :, 40] = -math.inf
    x[6, :, 31] = math.nan
    x[7] = -0.0
    x[8] = torch.linspace(-f.max, f.max, 64).to(dtype)
    x[9, :, :32] = torch.arange(32) * low
    x[10] = 1.0
    x[11, :, 1] = f.max
    x[11, :, 33] = -math.nan
    caches = [torch.full((3, 4, 1, 8 * bits), 0xA5, dtype=torch.uint8, device=DEV) for _ in "kv"]
    scales = [torch.full((3, 4, 1, 2), 0xA5, dtype=torch.uint8, device=DEV) for _ in "kv"]
    slots = torch.arange(12, dtype=torch.int32, device=DEV)
    y = x.to(DEV)
    vts.write_cache(y, y, y, slots, *caches, k_scales=scales[0], v_scales=scales[1])
    codes, scale = ref.quantise(x.double(), bits)
    for c, s in zip(caches, scales):
        assert torch.equal(s.cpu().view(12, 1, 2).long(), scale)
        got = ref.unpack(c.cpu().view(12, 1, -1), bits)
        assert torch.equal(ref.values(got, scale, bits).nan_to_num(5), ref.values(codes, scale, bits).nan_to_num(5))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim", [64, 128])
def test_read_every_code(bits, dim):
    """All bytes with scales from one end to the other, in bf16 and fp16: the numbers they stand
    for, rounded to nearest even."""
    scale = torch.tensor([0, 1, 2, 20, 100, 103, 110, 118, 126, 127, 128, 135, 142, 143, 160, 253, 254, 255])
    row = dim * bits // 8
    data = torch.arange(256).repeat(-(-len(scale) * 256 // 256)).to(torch.uint8)
    data = data.view(len(scale), 256 // row, 1, row) if row <= 256 else data
    k = data.to(DEV)
    s = scale.to(torch.uint8).view(-1, 1, 1, 1).expand(-1, 256 // row, 1, dim // 32).contiguous().to(DEV)
    slots = torch.arange(len(scale) * (256 // row), dtype=torch.int32, device=DEV)
    for dtype in (BF16, F16):
        got = vts.read_cache(k, k, slots, k_scales=s, v_scales=s, dtype=dtype)
        x = ref.values(ref.unpack(data, bits), s.cpu(), bits).view(-1, 1, dim)
        # (a number of the format has at most 4 bits, so fp32 holds it; one rounding)
        want = x.float().to(dtype)
        for y in got:
            y = y.cpu()
            assert torch.equal(y.isnan(), want.isnan())
            assert torch.equal(y[~y.isnan()], want[~want.isnan()])


def test_same_slot_read_many_times_and_none():
    gen = torch.Generator().manual_seed(1)
    (kc, vc), (ks, vs) = make_cache(gen, 3, 16, 3, 64, 4, None)
    slots = torch.tensor([[5, 5, 5], [47, -1, 48]], dtype=torch.int32, device=DEV)
    k, v = vts.read_cache(kc, vc, slots, k_scales=ks, v_scales=vs)
    assert k.shape == (2, 3, 3, 64) and k.dtype == BF16
    assert torch.equal(k[0, 0].view(torch.int16), k[0, 2].view(torch.int16))
    assert (k[1, 1:] == 0).all() and (v[1, 1:] == 0).all()
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert vts.read_cache(kc, vc, none, k_scales=ks, v_scales=vs)[0].shape == (0, 3, 64)
    q = torch.empty(0, 6, 64, dtype=BF16, device=DEV)
    before = kc.clone()
    out, kk = vts.write_cache(q, q[:, :3], q[:, :3], none, kc, vc, k_scales=ks, v_scales=vs, return_k=True)
    assert out.shape == (0, 6, 64) and kk.shape == (0, 3, 64) and torch.equal(kc, before)


def test_outputs_given_streams_and_graphs():
    gen = torch.Generator().manual_seed(2)
    q, k, v = make_tokens(gen, 40, 8, 2, 128, BF16)
    (kc, vc), (ks, vs) = make_cache(gen, 6, 16, 2, 128, 8, None)
    table = vts.rotary_table(100, 64, device=DEV)
    positions = torch.arange(40, dtype=torch.int32, device=DEV)
    slots = torch.randperm(96, generator=gen)[:40].int().to(DEV)
    w = torch.ones(128, device=DEV)
    kw = dict(k_scales=ks, v_scales=vs, positions=positions, rotary=table, q_norm=w, k_norm=w, return_k=True)
    want_q, want_k = vts.write_cache(q, k, v, slots, kc, vc, **kw)
    want = vts.read_cache(kc, vc, slots, k_scales=ks, v_scales=vs)
    torch.cuda.synchronize()
    out = torch.full((40, 8, 128), 3.0, dtype=BF16, device=DEV)
    side = torch.cuda.Stream()
    for t in (kc, vc, ks, vs):
        t.zero_()
    torch.cuda.synchronize()
    got, got_k = vts.write_cache(q, k, v, slots, kc, vc, q_out=out, stream=side, **kw)
    assert got is out
    back = vts.read_cache(kc, vc, slots, k_scales=ks, v_scales=vs, stream=side)
    side.synchronize()
    for a, b in ((got, want_q), (got_k, want_k), (back[0], want[0]), (back[1], want[1])):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gq, gk = vts.write_cache(q, k, v, slots, kc, vc, **kw)
        gr = vts.read_cache(kc, vc, slots, k_scales=ks, v_scales=vs)
    for turn in range(3):
        for t in (kc, vc, ks, vs):
            t.zero_()
        if turn == 2:  # new inputs in the same memory
            q.mul_(1.5)
            v.mul_(-1)
            want_q, want_k = vts.write_cache(q, k, v, slots, kc, vc, **kw)
            want = vts.read_cache(kc, vc, slots, k_scales=ks, v_scales=vs)
            kc.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((gq, want_q), (gk, want_k), (gr[0], want[0]), (gr[1], want[1])):
            assert torch.equal(a, b), turn


@pytest.mark.parametrize("bits", [4, 16])
def test_cache_past_4_gib(bits):
    """Slots whose rows lie beyond 2^32 bytes (and 2^31 elements)."""
    width = 64 if bits == 4 else 128
    pages = (5 << 30) // (64 * 8 * width * (1 if bits == 4 else 2))
    kind = torch.uint8 if bits == 4 else BF16
    kc, vc = (torch.empty(pages, 64, 8, width, dtype=kind, device=DEV) for _ in "kv")
    ks = vs = None
    if bits == 4:
        ks, vs = (torch.empty(pages, 64, 8, 4, dtype=torch.uint8, device=DEV) for _ in "kv")
    gen = torch.Generator().manual_seed(3)
    q, k, v = make_tokens(gen, 6, 8, 8, 128, BF16)
    n = pages * 64
    slots = torch.tensor([0, n - 1, n // 2, n - 64, n * 13 // 16, 5], dtype=torch.int32, device=DEV)
    vts.write_cache(q, k, v, slots, kc, vc, k_scales=ks, v_scales=vs)
    got = vts.read_cache(kc, vc, slots, k_scales=ks, v_scales=vs, dtype=BF16)
    for x, y in zip((k, v), got):
        if bits == 4:
            x = ref.values(*ref.quantise(x.cpu().double(), 4), 4).bfloat16()
        assert torch.equal(y.cpu(), x.cpu())


def test_gradients_are_none():
    q = torch.randn(2, 2, 64, device=DEV, dtype=BF16, requires_grad=True)
    c = torch.zeros(1, 16, 2, 64, device=DEV, dtype=BF16)
    slots = torch.arange(2, dtype=torch.int32, device=DEV)
    out, k = vts.write_cache(q, q, q, slots, c, c.clone(), return_k=True)
    assert not out.requires_grad and not k.requires_grad


def test_page_slots():
    table = torch.tensor([[3, 1, -1], [0, 2, 5]], dtype=torch.int32, device=DEV)
    pos = torch.tensor([[0, 17, 40, -1], [15, 16, 47, 48]], dtype=torch.int32, device=DEV)
    assert vts.page_slots(table, 16, pos).tolist() == [[48, 17, -1, -1], [15, 32, 95, -1]]


@pytest.mark.parametrize("bits", [4, 16])
def test_one_of_the_norms(bits):
    gen = torch.Generator().manual_seed(4)
    q, k, v = make_tokens(gen, 21, 6, 2, 64, BF16)
    (kc, vc), (ks, vs) = make_cache(gen, 3, 16, 2, 64, bits, BF16)
    w = torch.randn(64, generator=gen).to(DEV)
    slots = torch.arange(21, dtype=torch.int32, device=DEV)
    for qn, kn in ((w, None), (None, w)):
        got_q, got_k = vts.write_cache(q, k, v, slots, kc, vc, k_scales=ks, v_scales=vs, q_norm=qn, k_norm=kn,
                                       return_k=True)
        for got, x, n in ((got_q, q, qn), (got_k, k, kn)):
            y, m = ref.ready(x, n, 1e-6, None, None, False)
            assert ((got.cpu().double() - y).abs() <= ref.ready_bound(y, m, 64, BF16)).all()
            if n is None:
                assert torch.equal(got, x)


def test_infinities_and_nan_in_rows():
    """They stay in their row (and its pair), are kept by a 16-bit cache, and make a microscaled block
    NaN."""
    gen = torch.Generator().manual_seed(5)
    q, k, v = make_tokens(gen, 6, 4, 2, 64, BF16)
    q[1, 2, 40] = math.inf
    k[2, 1, 3] = math.nan
    v[3, 0, 33] = -math.inf
    table, slots = vts.rotary_table(64, 32, device=DEV), torch.arange(6, dtype=torch.int32, device=DEV)
    kw = dict(positions=slots, rotary=table, return_k=True)
    (kc, vc), _ = make_cache(gen, 1, 16, 2, 64, 16, BF16)
    got_q, got_k = vts.write_cache(q, k, v, slots, kc, vc, **kw)
    assert got_q[1, 2, 40] == math.inf and int((~got_q.isfinite()).sum()) == 1  # (not turned)
    bad = ~got_k.isfinite()
    assert bad[2, 1, 3] and bad[2, 1, 19] and int(bad.sum()) == 2
    assert torch.equal(at_slots(vc, slots).view(torch.int16), v.cpu().contiguous().view(torch.int16))
    (kc, vc), (ks, vs) = make_cache(gen, 1, 16, 2, 64, 8, BF16)
    vts.write_cache(q, k, v, slots, kc, vc, k_scales=ks, v_scales=vs, **kw)
    kk, vv = vts.read_cache(kc, vc, slots, k_scales=ks, v_scales=vs)
    assert kk[2, 1, :32].isnan().all() and int(kk.isnan().sum()) == 32
    assert vv[3, 0, 32:].isnan().all() and int(vv.isnan().sum()) == 32


def test_refusals():
    gen = torch.Generator().manual_seed(6)
    q, k, v = make_tokens(gen, 8, 4, 2, 64, BF16)
    (kc, vc), (ks, vs) = make_cache(gen, 2, 16, 2, 64, 4, BF16)
    (k16, v16), _ = make_cache(gen, 2, 16, 2, 64, 16, BF16)
    slots = torch.arange(8, dtype=torch.int32, device=DEV)
    table = vts.rotary_table(64, 32, device=DEV)
    mx = dict(k_scales=ks, v_scales=vs)
    own = torch.zeros(8, 4, 64, dtype=BF16, device=DEV)

    def write(q=q, k=k, v=v, slots=slots, kc=kc, vc=vc, **kw):
        vts.write_cache(q, k, v, slots, kc, vc, **{**mx, **kw})

    write()
    for match, kw in [
        ("k must", dict(k=k[:7])), ("k must", dict(k=k.float())), ("v must", dict(v=v[:, :1])),
        ("head_dim", dict(q=torch.zeros(8, 4, 128, dtype=BF16, device=DEV))), ("q rows", dict(q=q[..., :64:2])),
        ("slots", dict(slots=slots.long())), ("slots", dict(slots=slots.cpu())), ("slots", dict(slots=slots[:7])),
        ("together", dict(positions=slots)), ("together", dict(rotary=table)),
        ("rotary", dict(positions=slots, rotary=table.double())),
        ("rotary", dict(positions=slots, rotary=table[:, :24].contiguous())),
        ("rotary", dict(positions=slots, rotary=torch.zeros(9, 128, device=DEV))),
        ("positions", dict(positions=slots[:3], rotary=table)),
        ("q_norm", dict(q_norm=torch.ones(64, device=DEV).half())), ("k_norm", dict(k_norm=torch.ones(32, device=DEV))),
        ("eps", dict(eps=-1.0)), ("eps", dict(eps=math.nan)),
        ("q_out", dict(q_out=own[:7])), ("q_out", dict(q_out=own.float())),
        ("k_cache", dict(kc=k16)), ("shapes of K's|rows must be", dict(vc=vc[:, :, :1])),
        ("k_cache", dict(kc=kc[..., ::2])), ("together", dict(v_scales=None)),
        ("scales", dict(k_scales=ks[:1])), ("4-D uint8", dict(v_scales=vs.int())),
    ]:
        with pytest.raises(ValueError, match=match):
            write(**kw)
    with pytest.raises(ValueError, match="overlap"):
        vts.write_cache(own, k, v, slots, kc, vc, q_out=own, **mx)
    with pytest.raises(ValueError, match="own dtype"):
        vts.write_cache(q.half(), k, v, slots, k16, v16)
    with pytest.raises(ValueError, match="own dtype"):
        vts.read_cache(k16, v16, slots, dtype=F16)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        vts.read_cache(kc, vc, slots, dtype=torch.float32, **mx)
    for bad in (slots.long(), slots.cpu(), torch.arange(16, dtype=torch.int32, device=DEV)[::2], [1, 2]):
        with pytest.raises(ValueError, match="slots"):
            vts.read_cache(kc, vc, bad, **mx)
    cu = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    for match, args, kw in [
        ("cu_seqlens", (q, k, v, cu.long()), {}), ("cu_seqlens", (q, k, v, cu.cpu()), {}),
        ("cu_seqlens_k", (q, k, v, cu), dict(cu_seqlens_k=cu[:1])), ("dtype", (q.float(), k, v, cu), {}),
        ("k must", (q, k.half(), v, cu), {}), ("v must", (q, k, v[:7], cu), {}),
        ("multiple", (q[:, :3], k, v, cu), {}), ("out", (q, k, v, cu), dict(out=own[:7])),
        ("overlap", (own, k, v, cu), dict(out=own)), ("head_dim", (q[..., :32], k[..., :32], v[..., :32], cu), {}),
    ]:
        with pytest.raises(ValueError, match=match):
            vts.prompt_attention(*args, **kw)
    lens, pages = torch.tensor([8], dtype=torch.int32, device=DEV), torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    q4 = own.view(1, 8, 4, 64)
    for match, args, kw in [
        ("q dtype", (q4.float(), kc, vc, pages, lens), mx), ("k_cache", (q4, k16, v16, pages, lens), mx),
        ("k_cache dtype", (q4, kc, vc, pages, lens), {}), ("head_dim", (q4[..., :32], kc, vc, pages, lens), mx),
        ("together", (q4, kc, vc, pages, lens), dict(k_scales=ks)),
        ("overlap", (q4, kc, vc, pages, lens), dict(out=q4, **mx)),
    ]:
        with pytest.raises(ValueError, match=match):
            vts.tree_attention(*args, **kw)
