"""tree_attention where weights differ by many orders of magnitude, or are zero."""
import math

import pytest
import torch

import varlen_top_select_amd as vts
from tests import decode_ref as ref
from tests.test_gpu_decode import check_attend

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

DEV = "cuda"
# batch, kv, heads: every form of the workgroup
FORMS = [(1, 1, 4), (1, 1, 20), (32, 4, 16), (32, 4, 64), (32, 4, 80), (1, 2, 80), (1, 1, 100)]


def sinks(batch, kv, heads, dim, length, below, small, dtype, at):
    """One heavy place of small V, and `length - 1` places `below` nats under it with
    V = 1: equal scores, so 64 bits are two exponentials away."""
    page = 16
    width = -(-length // page)
    k = torch.zeros(batch * width, page, kv, dim, dtype=dtype, device=DEV)
    v = torch.ones_like(k)
    table = torch.arange(batch * width, dtype=torch.int32, device=DEV).view(batch, width)
    k[..., 0] = -below
    for b in range(batch):
        k[b * width + at // page, at % page, :, 0] = 0
        v[b * width + at // page, at % page] = small
    q = torch.zeros(batch, 1, heads, dim, dtype=dtype, device=DEV)
    q[..., 0] = 1
    lens = torch.full((batch,), length, dtype=torch.int32, device=DEV)
    out, lse = vts.tree_attention(q, k, v, table, lens, scale=1.0, return_lse=True)
    torch.cuda.synchronize()
    tail = (length - 1) * math.exp(-below)
    want = (float(torch.tensor(small, dtype=dtype)) + tail) / (1 + tail)
    return out.cpu().double(), lse.cpu().double(), want, math.log1p(tail)


@pytest.mark.parametrize("batch,kv,heads", FORMS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_light_places(batch, kv, heads, dim, dtype):
    """60000 places 17 nats under one whose V is small make up most of the output.
    A probability keeps half a step of relative error (eps / 2), the scores are
    exact, an exponent of 25 is held to 2^-20, the sums in 32 bits add 2^-24 a place
    and the output's rounding eps / 2."""
    length, below = 60001, 17.0
    out, lse, want, want_lse = sinks(batch, kv, heads, dim, length, below, 2.0 ** -13, dtype, length // 3)
    h = torch.finfo(dtype).eps / 2
    bound = want * (2 * h + 2.0 ** -19 + (length + 64) * 2.0 ** -24)
    worst = (out - want).abs().max().item()
    assert worst <= bound, f"{worst / bound:.3g} times the bound, want {want:.4g}"
    # the reference's bound of an lse: a sum is off by 2^-24 of itself at each place
    # (the heaviest place's weight, however little the others add)
    one = torch.ones(1, 1, 1, dtype=torch.float64)
    _, lb = ref.attend_bounds(one[..., None], one[..., None], below * one, length, dim, dtype)
    assert (lse - want_lse).abs().max().item() <= lb.item()


@pytest.mark.parametrize("batch,kv,heads", FORMS)
def test_lighter_places_in_fp16(batch, kv, heads):
    """22 nats under, past fp16's normal range: each place is off by half of fp16's
    least step, which lies 2^-36 of the heaviest weight at the most."""
    length = 60001
    out, _, want, _ = sinks(batch, kv, heads, 64, length, 22.0, 2.0 ** -14, torch.float16, 0)
    h = torch.finfo(torch.float16).eps / 2
    bound = want * (2 * h + 2.0 ** -19 + (length + 64) * 2.0 ** -24) + length * 2.0 ** -36 + 2.0 ** -25
    assert (out - want).abs().max().item() <= bound


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_climbing_scores(dtype):
    """The running maximum moves in small steps and in large ones, in every form."""
    gen = torch.Generator().manual_seed(70)
    for batch, kv, heads in FORMS:
        page, length, dim = 16, 900, 64
        width = -(-length // page)
        k, v = (torch.randn(batch * width, page, kv, dim, generator=gen).to(dtype).to(DEV) for _ in range(2))
        table = torch.arange(batch * width, dtype=torch.int32, device=DEV).view(batch, width)
        ramp = torch.cat([torch.linspace(0, 12, 400), torch.linspace(12, 60, 512)]).view(width, page, 1)
        k[..., 0] = ramp.repeat(batch, 1, 1).to(dtype).to(DEV)
        q = torch.randn(batch, 2, heads, dim, generator=gen).to(dtype).to(DEV)
        q[..., 0] = 1
        lens = torch.full((batch,), length, dtype=torch.int32, device=DEV)
        check_attend(q, k, v, table, lens, scale=0.5)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("batch,kv,heads", FORMS)
def test_nothing_of_weight(bad, batch, kv, heads):
    """Rows whose every score is -inf get zeros whatever V holds, the others what they see."""
    gen = torch.Generator().manual_seed(71)
    dim, page, length, dtype = 64, 16, 3000, torch.bfloat16
    width = -(-length // page)
    k, v = (torch.randn(batch * width, page, kv, dim, generator=gen).to(dtype).to(DEV) for _ in range(2))
    table = torch.arange(batch * width, dtype=torch.int32, device=DEV).view(batch, width)
    lens = torch.full((batch,), length, dtype=torch.int32, device=DEV)
    k[..., 0] = -math.inf
    v[..., 5] = bad
    q = torch.zeros(batch, 1, heads, dim, dtype=dtype, device=DEV)
    q[..., 0] = 1
    out, lse = vts.tree_attention(q, k, v, table, lens, return_lse=True)
    torch.cuda.synchronize()
    assert (lse == -math.inf).all()
    assert (out == 0).all()
    o64, l64, _, _ = ref.attend(q[:, :, :1], k[:, :, :1], v[:, :, :1], table, lens)
    assert (l64 == -math.inf).all() and (o64 == 0).all()
