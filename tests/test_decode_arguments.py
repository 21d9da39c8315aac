"""Arguments of the decode-step operators at their edges, without a GPU."""
import os

import pytest
import torch

import varlen_top_select_amd as vts
from varlen_top_select_amd import decode


@pytest.mark.parametrize("bad", [4, 5, 64, 2 ** 31 - 1, -2, -2 ** 31])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_tree_mask_of_parents_that_are_no_node(bad, dtype):
    """A node whose parent does not exist (verify_draft never accepts it) sees
    itself, and no entry past the row is looked up."""
    parents = torch.tensor([[-1, bad, 1, 0], [bad, 0, 1, bad]], dtype=dtype)
    assert vts.tree_mask_from_parents(parents).tolist() == [[1, 2, 6, 9], [1, 3, 7, 8]]


def test_tree_mask_of_no_tokens():
    assert vts.tree_mask_from_parents(torch.empty(3, 0, dtype=torch.int32)).shape == (3, 0)
    assert vts.tree_mask_from_parents(torch.empty(0, 5, dtype=torch.int32)).shape == (0, 5)


# ---- the C entry points, with pointers that are never dereferenced

OK, INVALID = 0, -1
A = 1 << 20  # fake, aligned "device" address


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(vts.LIB_PATH):
        from varlen_top_select_amd import build
        build.build()
    return vts.library()


def cache(batch=3, kv=4, dim=64, page=16):
    return decode._CACHE.pack(A, A, page * kv * dim, kv * dim, dim, page * kv * dim, kv * dim, dim, A,
                              100, 100, A, 50, page, kv, dim, batch, 1)


STRIDES = decode._STRIDES.pack(2 * 16 * 64, 16 * 64, 64)


@pytest.mark.parametrize("batch,kv,wb,wh,width,apart", [
    (3, 4, 400, 100, 100, True), (3, 4, 100, 300, 100, True),   # either order, nothing between
    (3, 4, 100, 100, 100, False),                               # row (0, 1) is row (1, 0)
    (3, 4, 300, 100, 100, False), (3, 4, 100, 250, 100, False),  # the last of one, the first of the next
    (3, 4, 399, 100, 100, False), (3, 4, 400, 99, 100, False), (3, 4, 99, 500, 100, False),
    (3, 4, 0, 100, 100, False), (3, 4, 400, 0, 100, False),
    (1, 4, 0, 100, 100, True), (3, 1, 100, 0, 100, True), (1, 1, 0, 0, 100, True),
    (2, 3, 300, 200, 100, True),    # 0 200 400 300 500 700: one within the other, apart
    (2, 3, 299, 200, 100, False), (3, 4, 150, 400, 100, True), (3, 4, 150, 399, 100, False),
    (3, 4, 1 << 62, 1 << 60, 100, True), (3, 4, (1 << 62) + 1, 1 << 61, 100, False),
])
def test_weights_rows_that_coincide(lib, batch, kv, wb, wh, width, apart):
    """Two rows that share an element would lose each other's additions."""
    rows = [b * wb + h * wh for b in range(batch) for h in range(kv)]
    assert apart == all(abs(x - y) >= width for i, x in enumerate(rows) for y in rows[:i])
    if apart and torch.cuda.is_available():
        pytest.skip("the call would run, on addresses that are none")
    got = lib.vts_attention_weight_add(cache(batch, kv), A, STRIDES, 2, 4 * kv, None, A, None, 0.1, A, wb,
                                       wh, width, None)
    assert (got != INVALID) == apart


def test_empty_batch_with_slots(lib):
    """The slots of no request: an address that is null and a top_k that is not 0."""
    def call(slots, top_k):
        return lib.vts_tree_attention(cache(batch=0), A, STRIDES, 2, 16, None, slots, top_k, 0.1, 2 * A,
                                      None, A, 1 << 40, None)
    assert call(None, 5) == call(None, 0) == call(A, 5) == OK
    assert call(A, 0) == INVALID and call(None, -1) == INVALID and call(A, -1) == INVALID


def strided(batch=3, kv=4, dim=64, page=16, pages=50, ks=None, vs=None):
    own = (page * kv * dim, kv * dim, dim)
    return decode._CACHE.pack(A, A, *(ks or own), *(vs or own), A, 100, 100, A, pages, page, kv, dim, batch, 1)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would run, on addresses that are none")
def test_strides_of_one_element_do_not_count(lib):
    """A dimension of one has no step: its stride may be anything."""
    big = 1 << 50

    def attend(c, q):
        return lib.vts_tree_attention(c, A, decode._STRIDES.pack(*q), 1 if q[1] == 3 else 2, 16, None, None,
                                      0, 0.1, 1 << 40, None, A, 1 << 40, None)
    plain = (2048, 1024, 64)
    own = (16 * 4 * 64, 4 * 64, 64)
    assert attend(strided(), plain) != INVALID
    assert attend(strided(kv=1, ks=(1024, 64, 1), vs=(1024, 64, big)), plain) != INVALID
    assert attend(strided(page=1, ks=(256, 7, 64), vs=(256, big, 64)), plain) != INVALID
    assert attend(strided(pages=1, ks=(3, 256, 64), vs=(big, 256, 64)), plain) != INVALID
    assert attend(strided(batch=1), (1, 1024, 64)) != INVALID
    assert attend(strided(), (2048, 3, 64)) != INVALID  # one drafted token
    # of two and more they do
    assert attend(strided(ks=(own[0], own[1], 4)), plain) == INVALID
    assert attend(strided(), (2044, 1024, 64)) == INVALID
    assert attend(strided(kv=1, ks=(1024, 60, 64)), plain) == INVALID
    assert attend(strided(), (2048, 1024, 4)) == INVALID


def test_binding_strides_of_one_element():
    t = torch.zeros(5, 3, 4, 64)
    assert decode._steps(t) == t.stride()[:3] == (768, 256, 64)
    one = torch.as_strided(t, (5, 3, 1, 64), (256, 64, 1, 1))
    assert decode._steps(one) == (256, 64, 0)
    assert decode._steps(torch.as_strided(t, (1, 3, 4, 64), (7, 256, 64, 1))) == (0, 256, 64)
    assert decode._steps(torch.as_strided(t, (1, 1, 1, 64), (3, 5, 1, 1))) == (0, 0, 0)
    for size, stride in (((5, 3, 4, 64), (768, 256, 60, 1)), ((5, 3, 1, 64), (256, 60, 64, 1))):
        assert decode._steps(torch.as_strided(t, size, stride)) is None
    column = torch.zeros(4, 6, dtype=torch.int32).t()[:, :1]  # one column of rows 1 apart
    assert column.stride() == (1, 6) and decode._row_step(column, 6) == 1
    assert decode._row_step(torch.zeros(6, 4).t(), 4) is None
    assert decode._row_step(torch.zeros(6, 4), 6) == 4
    assert decode._row_step(torch.zeros(1, 4), 1) == 4


def test_rows_that_meet_an_output():
    """Exactly the tensors with an element in the output's memory."""
    space = torch.zeros(6000, dtype=torch.bfloat16)
    gen = torch.Generator().manual_seed(5)

    def pick(*a):
        return a[int(torch.randint(len(a), (1,), generator=gen))]
    seen = [0, 0]
    for _ in range(6000):
        size = (pick(1, 2, 5), pick(1, 3), pick(1, 2, 4), pick(8, 16))
        stride = (pick(0, 8, 64, 200, 512), pick(8, 24, 64, 128, 300), pick(0, 8, 16, 40, 256), 1)
        t = space.as_strided(size, stride, pick(0, 8, 900, 2000))
        at = int(torch.randint(0, 5000, (1,), generator=gen))
        out = space[at:at + pick(1, 8, 64, 300)]
        mark = torch.zeros_like(space)
        mark.as_strided(size, stride, t.storage_offset()).fill_(1)
        want = bool(mark[at:at + out.numel()].any())
        assert decode._meets(out, t) == want, (size, stride, t.storage_offset(), at, out.numel())
        seen[want] += 1
    assert min(seen) > 300
    assert not decode._meets(space[:0], space.view(2, 3, 10, 100))
    assert not decode._meets(space, space.view(2, 3, 10, 100)[:0])


def test_no_kernel_that_no_call_reaches():
    """With a head to each wave there are at most 64 rows, which lie in registers or LDS."""
    if not os.path.exists(vts.LIB_PATH):
        from varlen_top_select_amd import build
        build.build()
    with open(vts.LIB_PATH, "rb") as f:
        names = f.read()
    for dtype in (1, 2):
        for dim in (64, 128):
            for heads in (0, 1):
                for rows in range(3):
                    name = f"weigh_kernelILi{dtype}ELi{dim}ELb{heads}ELi{rows}EE".encode()
                    assert (name in names) == (not (heads and rows == 2)), name
