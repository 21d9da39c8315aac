"""Refusals of the calls that fill and read a paged cache and attend prompts, and of the attention
over microscaled caches, without a GPU: the C entry points with pointers that are never dereferenced,
the binding's checks, and the plain helpers."""
import math
import os

import pytest
import torch

import varlen_top_select_amd as vts
from tests import cache_ref
from varlen_top_select_amd import cache as cache_mod, decode

OK, INVALID, UNSUPPORTED, WORKSPACE, HIP = 0, -1, -2, -3, -4
A = 1 << 20  # fake, aligned "device" address
BF16, F16, F32 = 1, 2, 0
NO_GPU = not torch.cuda.is_available()


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(vts.LIB_PATH):
        from varlen_top_select_amd import build
        build.build()
    return vts.library()


def cache(bits=16, **kw):
    w = 128 if bits == 16 else 16 * bits
    own = (64 * 8 * w, 8 * w, w)
    a = dict(k=A, v=A, ks=own, vs=own, table=A, stride=100, width=100, lens=A, pages=1000, page=64, kv=8,
             dim=128, batch=4, dtype=BF16)
    a.update(kw)
    return decode._CACHE.pack(a["k"] or 0, a["v"] or 0, *a["ks"], *a["vs"], a["table"] or 0,
                              a["stride"], a["width"], a["lens"] or 0, a["pages"], a["page"],
                              a["kv"], a["dim"], a["batch"], a["dtype"])


def scales(bits=4, **kw):
    a = dict(k=A, v=A, ks=(64 * 8 * 4, 8 * 4, 4), vs=(64 * 8 * 4, 8 * 4, 4), bits=bits)
    a.update(kw)
    return decode._SCALES.pack(a["k"] or 0, a["v"] or 0, *a["ks"], *a["vs"], a["bits"])


SCALE_ERRORS = [
    (dict(bits=16), INVALID), (dict(bits=0), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k=A + 2), INVALID), (dict(v=A + 1), INVALID), (dict(ks=(2048, 32, 2)), INVALID),
    (dict(vs=(-2048, 32, 4)), INVALID), (dict(ks=(1 << 40, 32, 4)), UNSUPPORTED),
    (dict(vs=(1 << 25, 32, 4)), UNSUPPORTED),  # past 2^32 rows at page 999
]
CACHE_ERRORS = [
    (dict(dtype=7), INVALID), (dict(dtype=F32), UNSUPPORTED), (dict(kv=0), INVALID), (dict(page=0), INVALID),
    (dict(pages=0), INVALID), (dict(dim=96), UNSUPPORTED), (dict(dim=0), INVALID), (dict(k=None), INVALID),
    (dict(v=A + 8), INVALID), (dict(ks=(64 * 8 * 128, 8 * 128, 4)), INVALID), (dict(vs=(-16, 16, 16)), INVALID),
    (dict(ks=(1 << 40, 1024, 128)), UNSUPPORTED), (dict(pages=1 << 40), UNSUPPORTED),
    (dict(page=(1 << 30) + 1), UNSUPPORTED),
]


def tokens(**kw):
    a = dict(q=A, k=A, v=A, qs=(48 * 128, 128), ks=(48 * 128, 128), vs=(48 * 128, 128), qn=A, kn=A, eps=1e-6,
             rotary=A, positions_max=100, positions=A, slots=A, n=10, out=2 * A, k_out=3 * A, heads=32,
             norm=BF16, rot=128, inter=0)
    a.update(kw)
    return cache_mod._TOKENS.pack(
        a["q"] or 0, a["k"] or 0, a["v"] or 0, *a["qs"], *a["ks"], *a["vs"], a["qn"] or 0, a["kn"] or 0,
        a["eps"], a["rotary"] or 0, a["positions_max"], a["positions"] or 0, a["slots"] or 0, a["n"],
        a["out"] or 0, a["k_out"] or 0, a["heads"], a["norm"], a["rot"], a["inter"])


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("kw,want", CACHE_ERRORS)
def test_write_and_read_refuse_caches(lib, kw, want, bits):
    m = None if bits == 16 else scales(bits)
    assert lib.vts_write_cache(cache(bits, **kw), m, tokens(), None) == want
    assert lib.vts_read_cache(cache(bits, **kw), m, A, 10, A, 2 * A, None) == want


@pytest.mark.parametrize("kw,want", SCALE_ERRORS)
def test_scales_are_refused(lib, kw, want):
    assert lib.vts_write_cache(cache(4), scales(**kw), tokens(), None) == want
    assert lib.vts_read_cache(cache(4), scales(**kw), A, 10, A, 2 * A, None) == want
    assert micro(lib, scales(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=A + 2), INVALID), (dict(qs=(-8, 8)), INVALID),
    (dict(ks=(48 * 128, 4)), INVALID), (dict(vs=(12, 128)), INVALID), (dict(n=-1), INVALID),
    (dict(heads=0), INVALID), (dict(heads=8193), UNSUPPORTED), (dict(n=(1 << 25) + 1), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(rot=8), INVALID), (dict(rot=24), INVALID), (dict(rot=144), INVALID), (dict(rot=0), INVALID),
    (dict(rotary=None), INVALID), (dict(rotary=A + 4), INVALID), (dict(positions_max=0), INVALID),
    (dict(positions_max=1 << 31), UNSUPPORTED), (dict(positions=None), INVALID), (dict(slots=None), INVALID),
    (dict(norm=F16), INVALID), (dict(norm=9), INVALID), (dict(qn=A + 8), INVALID), (dict(kn=A + 2), INVALID),
    (dict(out=None), INVALID), (dict(out=A + 4), INVALID), (dict(k_out=A + 4), INVALID),
    (dict(k_out=2 * A + 128), INVALID), (dict(n=0, q=None, slots=None, out=None), OK),
])
def test_write_refuses(lib, kw, want):
    assert lib.vts_write_cache(cache(), None, tokens(**kw), None) == want


def test_null_structures(lib):
    assert lib.vts_write_cache(None, None, tokens(), None) == INVALID
    assert lib.vts_write_cache(cache(), None, None, None) == INVALID
    assert lib.vts_read_cache(None, None, A, 10, A, 2 * A, None) == INVALID
    assert lib.vts_prompt_attention(None, 1, 1.0, A, None, 0, None, 0, None) == INVALID
    assert micro(lib, None) == INVALID


@pytest.mark.parametrize("slots,count,k,v,want", [
    (A, -1, A, 1 << 30, INVALID), (None, 10, A, 1 << 30, INVALID), (A, 10, None, 1 << 30, INVALID),
    (A, 10, A, None, INVALID), (A, 10, A + 8, 1 << 30, INVALID), (A, 10, A, A + 1024, INVALID),
    (A, 1 << 30, A, 1 << 50, UNSUPPORTED), (None, 0, None, None, OK),
])
def test_read_refuses(lib, slots, count, k, v, want):
    assert lib.vts_read_cache(cache(), None, slots, count, k, v, None) == want


def micro(lib, m, c=None, **kw):
    a = dict(q=A, draft=2, heads=64, mask=None, slots=None, top_k=0, scale=0.1, out=2 * A, lse=None,
             ws=A, bytes=1 << 40)
    a.update(kw)
    strides = decode._STRIDES.pack(2 * 64 * 128, 64 * 128, 128)
    return lib.vts_tree_attention_microscaled(c or cache(4), m, a["q"], strides, a["draft"], a["heads"],
                                              a["mask"], a["slots"], a["top_k"], a["scale"], a["out"], a["lse"],
                                              a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(draft=0), INVALID), (dict(draft=65), UNSUPPORTED), (dict(heads=63), INVALID), (dict(q=A + 2), INVALID),
    (dict(out=A + 8), INVALID), (dict(lse=2 * A + 16), INVALID), (dict(top_k=5), INVALID),
    (dict(slots=A), INVALID), (dict(scale=math.nan), INVALID), (dict(ws=None), WORKSPACE),
    (dict(bytes=100), WORKSPACE),
])
def test_micro_attention_refuses(lib, kw, want):
    assert micro(lib, scales(), **kw) == want
    assert micro(lib, scales(8), cache(8), **kw) == want


def test_micro_attention_refuses_tables(lib):
    for kw in (dict(batch=-1), dict(width=0), dict(stride=99), dict(table=None), dict(lens=None)):
        assert micro(lib, scales(), cache(4, **kw)) == INVALID
    assert micro(lib, scales(), cache(4, batch=0, table=None, lens=None)) == OK
    f = lib.vts_tree_attention_microscaled_workspace_bytes
    assert f(4, 2, 64, 8, 128, 0) > 65536 and f(4, 65, 64, 8, 128, 0) == 0 and f(4, 1, 63, 8, 128, 0) == 0


def prompts(**kw):
    a = dict(q=A, k=A, v=A, qs=(32 * 128, 128), ks=(8 * 128, 128), vs=(8 * 128, 128), cu_q=A, cu_k=A, batch=3,
             tq=100, tk=200, heads=32, kv=8, dim=128, dtype=BF16)
    a.update(kw)
    return cache_mod._PROMPTS.pack(a["q"] or 0, a["k"] or 0, a["v"] or 0, *a["qs"], *a["ks"], *a["vs"],
                                   a["cu_q"] or 0, a["cu_k"] or 0, a["batch"], a["tq"], a["tk"], a["heads"],
                                   a["kv"], a["dim"], a["dtype"])


@pytest.mark.parametrize("kw,call,want", [
    (dict(dtype=F32), {}, UNSUPPORTED), (dict(dtype=5), {}, INVALID), (dict(dim=80), {}, UNSUPPORTED),
    (dict(dim=0), {}, INVALID), (dict(batch=-1), {}, INVALID), (dict(tq=-1), {}, INVALID),
    (dict(tk=-1), {}, INVALID), (dict(kv=0), {}, INVALID), (dict(heads=33), {}, INVALID),
    (dict(heads=4), {}, INVALID), (dict(heads=16384), {}, UNSUPPORTED), (dict(tq=1 << 27), {}, UNSUPPORTED),
    (dict(tq=1 << 62), {}, UNSUPPORTED), (dict(tk=1 << 31), {}, UNSUPPORTED), (dict(batch=1 << 31), {}, UNSUPPORTED),
    (dict(q=None), {}, INVALID), (dict(k=A + 8), {}, INVALID), (dict(v=None), {}, INVALID),
    (dict(qs=(-8, 128)), {}, INVALID), (dict(ks=(8 * 128, 100)), {}, INVALID), (dict(cu_q=None), {}, INVALID),
    (dict(cu_k=None), {}, INVALID), ({}, dict(out=None), INVALID), ({}, dict(out=A + 8), INVALID),
    ({}, dict(lse=A + 2), INVALID), ({}, dict(out=A, lse=A + 256), INVALID), ({}, dict(scale=math.nan), INVALID),
    (dict(tq=4, tk=9000, batch=1), {}, WORKSPACE), (dict(tq=4, tk=9000, batch=1), dict(ws=A, bytes=100), WORKSPACE),
    (dict(tq=4, tk=9000, batch=1), dict(ws=A + 8, bytes=1 << 40), WORKSPACE),
    (dict(tq=0, q=None), dict(out=None), OK),
])
def test_prompt_refuses(lib, kw, call, want):
    a = dict(causal=1, scale=0.1, out=1 << 30, lse=None, clear=0, ws=None, bytes=0)
    a.update(call)
    assert lib.vts_prompt_attention(prompts(**kw), a["causal"], a["scale"], a["out"], a["lse"], a["clear"],
                                    a["ws"], a["bytes"], None) == want


def test_prompt_workspace(lib):
    """Only few queries behind long contexts take any; shapes that no call has take none."""
    f = lib.vts_prompt_attention_workspace_bytes
    assert f(1, 16384, 16384, 32, 8, 128) == 0 and f(1, 16, 1000, 32, 8, 128) == 0
    assert 0 < f(1, 16, 16384, 32, 8, 128) < 1 << 27
    assert f(1, 1, 1 << 30, 1, 1, 128) == f(1, 1, 1 << 20, 1, 1, 128) > 0
    for bad in ((-1, 1, 9000, 8, 8, 128), (1, -1, 9000, 8, 8, 128), (1, 1, 9000, 9, 8, 128), (1, 1, 9000, 8, 0, 128),
                (1, 1 << 62, 9000, 8, 8, 128), (1, 1, 9000, 1 << 30, 1, 128), (1, 1, 9000, 8, 8, 0)):
        assert f(*bad) == 0


def test_valid_calls_reach_the_device(lib):
    if NO_GPU:
        for got in (lib.vts_write_cache(cache(), None, tokens(), None),
                    lib.vts_read_cache(cache(4), scales(), A, 10, A, 1 << 30, None),
                    lib.vts_prompt_attention(prompts(), 1, 0.1, 1 << 30, None, 1, None, 0, None),
                    micro(lib, scales())):
            assert got in (HIP, UNSUPPORTED)


def test_binding_refuses():
    z = torch.zeros
    k = z(4, 16, 2, 64, dtype=torch.bfloat16)
    c8, s = z(4, 16, 2, 64, dtype=torch.uint8), z(4, 16, 2, 2, dtype=torch.uint8)
    x, slots = z(3, 2, 64, dtype=torch.bfloat16), z(3, dtype=torch.int32)
    table, lens = z(1, 4, dtype=torch.int32), z(1, dtype=torch.int32)
    for bad in (z(4, 16, 128), k.float(), None, k):  # the last one: not on the GPU
        with pytest.raises(ValueError, match="k_cache"):
            vts.write_cache(x, x, x, slots, bad, bad)
        with pytest.raises(ValueError, match="k_cache"):
            vts.read_cache(bad, bad, slots)
    with pytest.raises(ValueError, match="together"):
        vts.read_cache(c8, c8, slots, k_scales=s)
    with pytest.raises(ValueError, match="together"):
        vts.tree_attention(x.view(1, 3, 2, 64), c8, c8, table, lens, v_scales=s)
    with pytest.raises(ValueError, match="k_cache"):
        vts.tree_attention(x.view(1, 3, 2, 64), c8, c8, table, lens, k_scales=s, v_scales=s)
    with pytest.raises(ValueError, match="q must"):
        vts.write_cache(None, x, x, slots, k, k)
    for bad in (None, x):
        with pytest.raises(ValueError, match="GPU"):
            vts.prompt_attention(bad, x, x, lens)
    for kw in (dict(max_position=0, rot=64), dict(max_position=10, rot=24), dict(max_position=10, rot=0)):
        with pytest.raises(ValueError, match="rot"):
            vts.rotary_table(**kw)
    with pytest.raises(ValueError, match="positions"):
        vts.page_slots(table, 16, lens)


def test_rotary_table():
    t = vts.rotary_table(200000, 64, base=500000.0)
    assert t.shape == (200000, 64) and t.dtype == torch.float32
    for p, i in ((0, 0), (199999, 0), (131071, 7), (1, 31)):
        angle = p * 500000.0 ** (-2 * i / 64)
        assert abs(float(t[p, i]) - math.cos(angle)) < 1e-7 and abs(float(t[p, 32 + i]) - math.sin(angle)) < 1e-7


def test_page_slots():
    table = torch.tensor([[3, 1, -1], [0, 2, 5]], dtype=torch.int32)
    pos = torch.tensor([[0, 17, 40, -1], [15, 16, 47, 48]])
    assert vts.page_slots(table, 16, pos).tolist() == [[48, 17, -1, -1], [15, 32, 95, -1]]
    assert vts.page_slots(table, 16, pos.int()).dtype == torch.int32


def test_page_slots_at_the_ends():
    """Entries whose slots pass 32 bits (2^28 + 3 pages of 16 came back as page 3), and tables
    without columns."""
    pos = torch.tensor([[5], [5], [15]])
    table = torch.tensor([[2**28 + 3], [2**27], [2**27 - 1]], dtype=torch.int32)
    assert vts.page_slots(table, 16, pos).tolist() == [[-1], [-1], [2**31 - 1]]
    assert vts.page_slots(table[:, :0], 16, pos).tolist() == [[-1], [-1], [-1]]
    assert vts.page_slots(table[:0], 16, pos[:0]).shape == (0, 1)
    with pytest.raises(ValueError, match="page_size"):
        vts.page_slots(table, 0, pos)


@pytest.mark.parametrize("bits", [4, 8])
def test_reference_formats(bits):
    """The oracle's numbers: every value is its own nearest, ties go to the even code, and the
    scale is the least that holds the largest."""
    n = cache_ref.numbers(bits)
    assert float(n[-1]) == (6 if bits == 4 else 448) and len(n) == (8 if bits == 4 else 127)
    if bits == 8:
        assert torch.equal(n, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double())
        x = torch.linspace(0, 463, 5000, dtype=torch.float64)
        assert torch.equal(n[cache_ref.nearest(x, n)].float(), x.float().to(torch.float8_e4m3fn).float())
    assert torch.equal(cache_ref.nearest(n, n), torch.arange(len(n)))
    mids = (n[1:] + n[:-1]) / 2
    assert (cache_ref.nearest(mids, n) % 2 == 0).all()
    for top, e in ((6.0, 0), (6.99, 0), (7.0, 1), (3.5, 0), (3.4, -1)) if bits == 4 else (
            (448.0, 0), (464.0, 0), (464.01, 1), (232.0, -1)):
        x = torch.zeros(1, 32, dtype=torch.float64)
        x[0, 7] = -top
        codes, scale = cache_ref.quantise(x, bits)
        assert int(scale) == 127 + e
        assert abs(float(cache_ref.values(codes, scale, bits)[0, 7]) + top) <= 2.0 ** e * (1 if bits == 4 else 16)
