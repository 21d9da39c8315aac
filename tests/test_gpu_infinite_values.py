"""Infinities in V count with the weight of their key, wherever a tile ends: a key whose score is
-inf has none, and 0 times an infinity is NaN.  Decoding over microscaled caches in fp16."""
import math

import pytest
import torch

from tests import cache_ref, decode_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_micro_attention import F16, DEV, make_cache, say  # noqa: E402
from tests.test_gpu_micro_not_finite import DENSE, PAGE, infinite, place, run  # noqa: E402


def same_kind(got, want):
    """The infinities and NaN of the 64-bit form, and nothing else that is not finite."""
    got, want = got.cpu().double(), want.cpu().double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got == math.inf, want == math.inf)
    assert torch.equal(got == -math.inf, want == -math.inf)


def within(got, o64, ob):
    """The finite outputs are within the bound."""
    ok = o64.isfinite()
    worst = ((got.cpu().double() - o64).abs() / ob)[ok].max().item()
    assert worst <= 1, f"output {worst:.3g} times its bound"


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("draft,heads,kv,batch", DENSE)
def test_scores_of_minus_infinity(draft, heads, kv, batch, bits):
    """Places seen with a score of -inf, among the drafted tokens, at the prefix's end and further back;
    their V's infinities give NaN."""
    say("scores", draft, heads, kv, batch, bits)
    gen = torch.Generator().manual_seed(910)
    lens = ([70 + draft, 101 + draft, 130 + draft] * batch)[:batch]
    caches, scales, deep, table, n = make_cache(gen, lens, PAGE, kv, 128, bits)
    q = (0.2 * torch.randn(batch, draft, heads, 128, generator=gen)).half()
    q[..., :32] = q[..., :32].abs() + 0.01
    q = q.to(DEV)
    for i, spots in enumerate(((70, 69), (100, 5), (131, 40))):
        for j, pos in enumerate(spots):
            at = place(table, i, pos)
            infinite(caches, scales, bits, 0, at, 0, -1)
            infinite(caches, scales, bits, 1, at, 1 + j, 1)
    deep = [cache_ref.values(cache_ref.unpack(c.cpu(), bits), s.cpu(), bits).half() for c, s in zip(caches, scales)]
    got, lse = run(q, caches, scales, table, n)
    few = slice(0, 3)
    tame = [d.clone().nan_to_num(0, 0, 0) for d in deep]
    _, _, _, reach = ref.attend(q[few], *tame, table[few], n[few])
    o64, l64, mag, _ = ref.attend(q[few], *deep, table[few], n[few])
    assert o64[:, :, :, 32:].isnan().any() and l64.isfinite().all()
    same_kind(got[few], o64)
    ob, lb = ref.attend_bounds(o64.nan_to_num(0, 0, 0), mag.nan_to_num(0, 0, 0), reach, max(lens), 128, F16)
    within(got[few], o64, ob)
    assert ((lse[few].double() - l64).abs() <= lb).all()
    assert got[3:].isfinite().all()
