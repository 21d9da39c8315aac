"""Refusals of the decode-step operators, without a GPU: the C entry points with
pointers that are never dereferenced, and the binding's checks."""
import os

import pytest
import torch

import varlen_top_select_amd as vts
from varlen_top_select_amd import decode

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


def cache(**kw):
    a = dict(k=A, v=A, ks=(64 * 8 * 128, 8 * 128, 128), vs=(64 * 8 * 128, 8 * 128, 128), table=A,
             stride=100, width=100, lens=A, pages=1000, page=64, kv=8, dim=128, batch=4, dtype=BF16)
    a.update(kw)
    return decode._CACHE.pack(a["k"] or 0, a["v"] or 0, *a["ks"], *a["vs"], a["table"] or 0,
                              a["stride"], a["width"], a["lens"] or 0, a["pages"], a["page"],
                              a["kv"], a["dim"], a["batch"], a["dtype"])


STRIDES = decode._STRIDES.pack(2 * 64 * 128, 64 * 128, 128)
CACHE_ERRORS = [
    (dict(dtype=7), INVALID), (dict(dtype=F32), UNSUPPORTED), (dict(batch=-1), INVALID),
    (dict(kv=0), INVALID), (dict(page=0), INVALID), (dict(pages=0), INVALID),
    (dict(width=0), INVALID), (dict(stride=99), INVALID), (dict(dim=96), UNSUPPORTED),
    (dict(dim=0), INVALID), (dict(kv=7), INVALID), (dict(k=None), INVALID),
    (dict(k=A + 8), INVALID), (dict(ks=(64 * 8 * 128, 8 * 128, 4)), INVALID),
    (dict(ks=(-8, 8, 8)), INVALID), (dict(ks=(1 << 40, 1024, 128)), UNSUPPORTED),
    (dict(ks=(1 << 30, 1024, 128)), UNSUPPORTED),  # past 2^32 vectors at page 999
    (dict(pages=1 << 40), UNSUPPORTED), (dict(page=(1 << 30) + 1), UNSUPPORTED),
    (dict(table=None), INVALID), (dict(lens=None), INVALID),
]


def attention(lib, c=None, **kw):
    a = dict(q=A, draft=2, heads=64, mask=None, slots=None, top_k=0, scale=0.1, out=2 * A, lse=None,
             ws=A, bytes=1 << 40)
    a.update(kw)
    return lib.vts_tree_attention(c or cache(), a["q"], STRIDES, a["draft"], a["heads"], a["mask"],
                                  a["slots"], a["top_k"], a["scale"], a["out"], a["lse"], a["ws"],
                                  a["bytes"], None)


@pytest.mark.parametrize("kw,want", CACHE_ERRORS + [(dict(v=None), INVALID), (dict(v=A + 2), INVALID)])
def test_attention_refuses_caches(lib, kw, want):
    assert attention(lib, cache(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(draft=0), INVALID), (dict(draft=65), UNSUPPORTED), (dict(heads=4), INVALID),
    (dict(heads=63), INVALID), (dict(q=None), INVALID), (dict(q=A + 2), INVALID),
    (dict(out=None), INVALID), (dict(out=A + 8), INVALID), (dict(lse=A + 2), INVALID),
    (dict(lse=2 * A + 16), INVALID), (dict(top_k=5), INVALID), (dict(slots=A), INVALID),
    (dict(slots=A, top_k=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=A + 4), WORKSPACE), (dict(bytes=100), WORKSPACE),
])
def test_attention_refuses(lib, kw, want):
    assert attention(lib, **kw) == want


def test_attention_empty_batch_and_null_cache(lib):
    assert attention(lib, cache(batch=0, table=None, lens=None)) == OK
    assert lib.vts_tree_attention(None, A, STRIDES, 1, 64, None, None, 0, 1.0, A, None, A, 1 << 40,
                                  None) == INVALID
    if NO_GPU:
        assert attention(lib) in (HIP, UNSUPPORTED)


def test_attention_workspace_is_a_function_of_the_shape(lib):
    f = lib.vts_tree_attention_workspace_bytes
    assert f(4, 2, 64, 8, 128, 0) == f(4, 2, 64, 8, 128, 0) > 65536
    assert f(4, 0, 64, 8, 128, 0) == 0 and f(4, 65, 64, 8, 128, 0) == 0
    assert f(4, 1, 63, 8, 128, 0) == 0 and f(-1, 1, 64, 8, 128, 0) == 0
    for draft, heads, kv in ((64, 512, 1), (1, 1, 1), (64, 8192, 1), (16, 64, 8)):
        assert 0 < f(4, draft, heads, kv, 128, 0) < 1 << 32


def weigh(lib, c=None, **kw):
    a = dict(q=A, draft=2, heads=64, lse=A, scale=0.1, w=A, wb=800, wh=100, width=100)
    a.update(kw)
    return lib.vts_attention_weight_add(c or cache(), a["q"], STRIDES, a["draft"], a["heads"], None,
                                        a["lse"], None, a["scale"], a["w"], a["wb"], a["wh"],
                                        a["width"], None)


@pytest.mark.parametrize("kw,want", CACHE_ERRORS)
def test_weigh_refuses_caches(lib, kw, want):
    assert weigh(lib, cache(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(draft=0), INVALID), (dict(draft=65), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(lse=None), INVALID), (dict(w=None), INVALID), (dict(w=A + 2), INVALID),
    (dict(wb=-1), INVALID), (dict(width=-1), INVALID), (dict(width=0), OK),
    (dict(scale=float("nan")), INVALID),
])
def test_weigh_refuses(lib, kw, want):
    assert weigh(lib, **kw) == want


def evict(lib, c=None, **kw):
    a = dict(w=A, wb=800, wh=100, width=100, keep=640, sinks=4, recent=30, ko=A, vo=A, pages=40,
             table=A, stride=10, twidth=10, kept=A, lens=A, ow=2 * A, os=(64 * 8 * 128, 8 * 128, 128))
    a.update(kw)
    s = decode._STRIDES.pack(*a["os"])
    return lib.vts_evict_cache(c or cache(), a["w"], a["wb"], a["wh"], a["width"], a["keep"],
                               a["sinks"], a["recent"], a["ko"], s, a["vo"], s, a["pages"],
                               a["table"], a["stride"], a["twidth"], a["kept"], a["lens"], a["ow"],
                               None)


@pytest.mark.parametrize("kw,want", [c for c in CACHE_ERRORS if c[0] != dict(kv=7)])
def test_evict_refuses_caches(lib, kw, want):
    assert evict(lib, cache(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(keep=0), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID),
    (dict(sinks=320, recent=321), INVALID), (dict(width=0), INVALID), (dict(pages=0), INVALID),
    (dict(twidth=9), INVALID), (dict(stride=9), INVALID), (dict(ko=None), INVALID),
    (dict(vo=A + 2), INVALID), (dict(os=(64, 4, 8)), INVALID), (dict(w=None), INVALID),
    (dict(table=None), INVALID), (dict(kept=None), INVALID), (dict(lens=None), INVALID),
    (dict(ow=None), INVALID), (dict(ow=A + 64), INVALID),
    (dict(keep=1 << 30, twidth=1 << 24, stride=1 << 24), UNSUPPORTED),
])
def test_evict_refuses(lib, kw, want):
    assert evict(lib, **kw) == want


def verify(lib, **kw):
    a = dict(p=A, dtype=F32, tb=4000, tr=1000, q=A, qb=3000, qr=1000, tokens=A, parents=None, u=A,
             batch=4, draft=3, vocab=1000, path=A, count=A, token=A, ws=A, bytes=1 << 40)
    a.update(kw)
    return lib.vts_verify_draft(a["p"], a["dtype"], a["tb"], a["tr"], a["q"], a["qb"], a["qr"],
                                a["tokens"], a["parents"], a["u"], a["batch"], a["draft"],
                                a["vocab"], a["path"], a["count"], a["token"], a["ws"], a["bytes"],
                                None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), INVALID), (dict(batch=-1), INVALID), (dict(draft=0), INVALID),
    (dict(draft=65), UNSUPPORTED), (dict(vocab=0), INVALID), (dict(vocab=1 << 31), UNSUPPORTED),
    (dict(tb=-1), INVALID), (dict(qr=-1), INVALID), (dict(p=None), INVALID), (dict(p=A + 2), INVALID),
    (dict(q=A + 1), INVALID), (dict(tokens=None), INVALID), (dict(u=None), INVALID),
    (dict(path=None), INVALID), (dict(count=None), INVALID), (dict(token=None), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=A + 8), WORKSPACE), (dict(bytes=64), WORKSPACE),
    (dict(batch=0), OK), (dict(batch=(1 << 21) + 1), UNSUPPORTED),
])
def test_verify_refuses(lib, kw, want):
    assert verify(lib, **kw) == want


def test_binding_refuses():
    z = torch.zeros
    k = z(4, 16, 2, 64, dtype=torch.bfloat16)
    table, lens = z(1, 4, dtype=torch.int32), z(1, dtype=torch.int32)
    q = z(1, 1, 2, 64, dtype=torch.bfloat16)
    for bad in (z(4, 16, 128), k.float(), None, k):  # the last one: not on the GPU
        with pytest.raises(ValueError, match="k_cache"):
            vts.tree_attention(q, bad, bad, table, lens)
        with pytest.raises(ValueError, match="k_cache"):
            vts.attention_weight_add(z(1, 2, 64), q, bad, table, lens, z(1, 1, 2))
        with pytest.raises(ValueError, match="k_cache"):
            vts.evict_cache(z(1, 2, 64), bad, bad, table, lens, 16, k, k, table)
    for bad in (z(2, 5), z(1, 2, 5, dtype=torch.int32), z(1, 2, 5)):
        with pytest.raises(ValueError, match="target_probs"):
            vts.verify_draft(bad, z(1, 1, dtype=torch.int32), z(1, 2))
    with pytest.raises(ValueError, match="parents"):
        vts.tree_mask_from_parents(z(1, 65, dtype=torch.int32))


def test_tree_mask():
    parents = torch.tensor([[-1, 0, 0, 1, 3, 2, 4], [-1, -1, -1, -1, -1, -1, 5]], dtype=torch.int32)
    want = []
    for row in parents.tolist():
        bits = []
        for t, p in enumerate(row):
            bits.append((bits[p] if p >= 0 else 0) | 1 << t)
        want.append(bits)
    assert vts.tree_mask_from_parents(parents).tolist() == want
    chain = (torch.arange(64) - 1).view(1, 64).int()
    got = vts.tree_mask_from_parents(chain)[0].tolist()
    assert [x & (1 << 64) - 1 for x in got] == [(2 << t) - 1 for t in range(64)]
