"""tree_attention over 16-bit caches with infinities in V of places that rows see: those of keys with a
score of -inf give NaN, those of weight themselves, next to drafted tokens and further back."""
import math

import pytest
import torch

import varlen_top_select_amd as vts
from tests import decode_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_infinite_values import same_kind, within  # noqa: E402
from tests.test_gpu_micro_attention import BF16, DEV, F16, say  # noqa: E402
from tests.test_gpu_micro_not_finite import DENSE, PAGE, place  # noqa: E402


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("draft,heads,kv,batch", DENSE)
def test_scores_of_minus_infinity(draft, heads, kv, batch, dtype):
    say("16 bits", draft, heads, kv, batch, dtype)
    gen = torch.Generator().manual_seed(950)
    lens = ([70 + draft, 101 + draft, 130 + draft] * batch)[:batch]
    width = max(-(-n // PAGE) for n in lens)
    table = torch.randperm(batch * width, generator=gen).view(batch, width).int().to(DEV)
    k, v = (torch.randn(batch * width, PAGE, kv, 128, generator=gen).to(dtype) for _ in "kv")
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = (0.2 * torch.randn(batch, draft, heads, 128, generator=gen)).to(dtype)
    q[..., 5] = q[..., 5].abs() + 0.01
    q = q.to(DEV)
    tame = k.clone()
    for i, spots in enumerate(((70, 69), (100, 5), (131, 40))):
        for j, pos in enumerate(spots):
            page, at = place(table, i, pos)
            k[page, at, :, 5], tame[page, at, :, 5] = -math.inf, 0
            v[page, at, :, 10 + j] = math.inf
        page, at = place(table, i, (69, 100, 20)[i])  # and of weight (request 0's has none)
        v[page, at, :, 40 + i] = -math.inf
    got, lse = vts.tree_attention(q, k.to(DEV), v.to(DEV), table, n, return_lse=True)
    few = slice(0, 3)
    o64, l64, mag, _ = ref.attend(q[few], k, v, table[few], n[few])
    _, _, _, reach = ref.attend(q[few], tame, v, table[few], n[few])
    assert o64.isnan().any() and (o64 == -math.inf).any()
    same_kind(got[few], o64)
    ob, lb = ref.attend_bounds(o64.nan_to_num(0, 0, 0), mag.nan_to_num(0, 0, 0), reach, max(lens), 128, dtype)
    within(got[few], o64, ob)
    assert ((lse[few].cpu().double() - l64).abs() <= lb).all()
    assert got[3:].isfinite().all()
