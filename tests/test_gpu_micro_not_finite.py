"""tree_attention over microscaled caches whose V holds NaN or infinities in places that rows see:
in the tile that the end of a list shares with the drafted tokens and in earlier ones, for every
form of workgroup, dense and with slot lists."""
import math

import pytest
import torch

import varlen_top_select_amd as vts

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_micro_attention import BF16, DEV, F16, make_cache, random_mask, say  # noqa: E402

PAGE = 16


def run(q, caches, scales, table, n, mask=None, slots=None):
    out, lse = vts.tree_attention(q, *caches, table, n, tree_mask=mask, slots=slots, k_scales=scales[0],
                                  v_scales=scales[1], return_lse=True)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def place(table, b, pos):
    return int(table[b, pos // PAGE]), pos % PAGE


def infinite(caches, scales, bits, which, at, block, sign=1):
    """A block of numbers past fp16's range."""
    code = {8: 0x70, 4: 0x77}[bits] | (0 if sign > 0 else {8: 0x80, 4: 0x88}[bits])  # 128, 6 and 6
    width = 32 * bits // 8
    caches[which][at[0], at[1], :, block * width:(block + 1) * width] = code
    scales[which][at[0], at[1], :, block] = 127 + 14


# draft, heads, kv, requests: 16 and 32 rows to a workgroup of one head, to a wave of four heads,
# and wide workgroups of 64 and 128 rows
DENSE = [(3, 8, 2, 3), (8, 8, 2, 3), (4, 16, 4, 33), (8, 16, 4, 33), (16, 8, 2, 3), (40, 8, 2, 3)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("draft,heads,kv,batch", DENSE)
def test_values_of_the_prefix(draft, heads, kv, batch, dtype, bits):
    """NaN in V's blocks of the prefix's last place and of one further back: NaN in those elements of
    every row of the request, and nothing else changes.  In fp16 also infinities."""
    say("prefix", draft, heads, kv, batch, dtype, bits)
    gen = torch.Generator().manual_seed(900)
    # (the prefix ends inside a tile of 32, with the draft behind it)
    lens = ([70 + draft, 101 + draft, 130 + draft] * batch)[:batch]
    caches, scales, deep, table, n = make_cache(gen, lens, PAGE, kv, 128, bits)
    q = (0.2 * torch.randn(batch, draft, heads, 128, generator=gen)).to(dtype).to(DEV)
    mask = random_mask(gen, batch, draft)
    clean, clean_lse = run(q, caches, scales, table, n, mask)
    assert clean.isfinite().all()
    for i, (last, back) in enumerate(((69, 5), (100, 64), (129, 40))):
        for pos, block in ((last, 2), (back, 0)):
            page, at = place(table, i, pos)
            scales[1][page, at, :, block] = 255
        if dtype == F16:
            infinite(caches, scales, bits, 1, place(table, i, last), 3, -1)
    got, lse = run(q, caches, scales, table, n, mask)
    assert torch.equal(lse, clean_lse)
    for i in range(3):
        assert got[i, :, :, 64:96].isnan().all(), i
        assert got[i, :, :, :32].isnan().all(), i
        assert torch.equal(got[i, :, :, 32:64], clean[i, :, :, 32:64])
        if dtype == F16:
            assert (got[i, :, :, 96:] == -math.inf).all(), i
        else:
            assert torch.equal(got[i, :, :, 96:], clean[i, :, :, 96:])
    assert torch.equal(got[3:], clean[3:])


# draft, heads, kv, requests, the list's length
LISTS = [(2, 8, 2, 3, 70), (1, 40, 2, 3, 33), (2, 16, 4, 17, 70), (1, 128, 4, 33, 41), (2, 96, 2, 3, 75),
         (1, 200, 2, 3, 100), (1, 8, 2, 3, 1)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("draft,heads,kv,batch,top_k", LISTS)
def test_values_of_listed_slots(draft, heads, kv, batch, top_k, tree, bits):
    say("slots", draft, heads, kv, batch, top_k, tree, bits)
    gen = torch.Generator().manual_seed(901)
    lens = ([50, 90, 33] * batch)[:batch]
    caches, scales, deep, table, n = make_cache(gen, lens, PAGE, kv, 128, bits)
    pages = caches[0].shape[0]
    used = set(table.cpu().flatten().tolist())
    spare = [x for x in range(pages) if x not in used]  # pages of nobody
    known = torch.tensor(sorted(used - {-1})).int()
    slots = known[torch.randint(0, len(known), (batch, draft, top_k), generator=gen)] * PAGE
    slots += torch.randint(0, PAGE, slots.shape, generator=gen)
    q = (0.2 * torch.randn(batch, draft, heads, 128, generator=gen)).bfloat16().to(DEV)
    mask = random_mask(gen, batch, draft) if tree else None
    slots[0, :, -1] = spare[0] * PAGE + 3
    slots[1, :, 0] = spare[1] * PAGE + 7
    slots = slots.int().to(DEV)
    clean, clean_lse = run(q, caches, scales, table, n, mask, slots)
    assert clean.isfinite().all()
    scales[1][spare[0], 3, :, 1] = 255
    scales[1][spare[1], 7, :, 3] = 255
    got, lse = run(q, caches, scales, table, n, mask, slots)
    assert torch.equal(lse, clean_lse)
    assert got[0, :, :, 32:64].isnan().all() and got[1, :, :, 96:].isnan().all()
    got[0, :, :, 32:64], got[1, :, :, 96:] = clean[0, :, :, 32:64], clean[1, :, :, 96:]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("heads", [2, 6])
def test_infinities_of_places_that_part_of_a_workgroup_sees(heads, bits):
    """Rows that see drafted tokens 32 and more alone, of which one is infinite: the waves of the first
    32 places see nothing of those rows."""
    draft = 40
    gen = torch.Generator().manual_seed(911)
    caches, scales, deep, table, n = make_cache(gen, [draft, draft], PAGE, 2, 128, bits)
    q = (0.2 * torch.randn(2, draft, heads, 128, generator=gen)).half().to(DEV)
    mask = torch.tensor([1 << t | (1 << 33 if t >= 32 else 0) for t in range(draft)]).expand(2, -1).contiguous().to(DEV)
    clean, clean_lse = run(q, caches, scales, table, n, mask)
    infinite(caches, scales, bits, 1, place(table, 1, 33), 2)
    got, lse = run(q, caches, scales, table, n, mask)
    assert torch.equal(lse, clean_lse)
    assert (got[1, 32:, :, 64:96] == math.inf).all()
    got[1, 32:, :, 64:96] = clean[1, 32:, :, 64:96]
    assert torch.equal(got, clean)
