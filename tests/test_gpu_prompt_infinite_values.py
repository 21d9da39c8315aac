"""prompt_attention with infinities in V of keys that rows see: those of keys with a score of -inf give
NaN (0 times an infinity) and those of weight themselves, in tiles that every row sees and in others."""
import math

import pytest
import torch

import varlen_top_select_amd as vts
from tests import cache_ref, decode_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_infinite_values import same_kind, within  # noqa: E402
from tests.test_gpu_micro_attention import BF16, F16, say  # noqa: E402
from tests.test_gpu_prompt import tensors  # noqa: E402

PROMPTS = [
    # query lengths, keys in front, heads, kv, dim, causal
    ([300, 40], [0, 0], 4, 2, 128, True),
    ([200, 3], [150, 70], 14, 2, 64, True),
    ([70, 130], [9, 0], 4, 4, 64, False),
    ([16], [3300], 4, 2, 128, True),        # keys shared by workgroups
    ([16, 40], [2500, 1100], 8, 2, 64, False),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("i", range(len(PROMPTS)))
def test_prompts(i, dtype):
    """Keys that rows see with a score of -inf, in tiles that every row sees and in the last ones."""
    lens, front, heads, kv, dim, causal = PROMPTS[i]
    say("prompt", PROMPTS[i], dtype)
    gen = torch.Generator().manual_seed(920 + i)
    q, k, v, cu_q, cu_k = tensors(gen, lens, front, heads, kv, dim, dtype)
    q[..., 5] = q[..., 5].abs() + 0.01
    ends = cu_k.tolist()
    spots = [3, 70, lens[0] + front[0] - 2, ends[1] - 40] + ([ends[1] + 1, ends[2] - 3] if len(lens) > 1 else [])
    tame = k.clone()
    for n, j in enumerate(spots):
        k[j, :, 5] = -math.inf
        tame[j, :, 5] = 0
        v[j, 0, 2 * n] = math.inf
        v[j, -1, 2 * n + 1] = -math.inf
    # and of weight
    v[20, 0, 40] = math.inf
    v[ends[1] - 1, -1, 41] = -math.inf
    v[ends[1] - 7, 0, 42] = math.nan
    got, lse = vts.prompt_attention(q, k, v, cu_q, cu_seqlens_k=cu_k, causal=causal, return_lse=True)
    o64, l64, mag, _ = cache_ref.prompt(q, k, v, cu_q, cu_k, causal)
    _, _, _, reach = cache_ref.prompt(q, tame, v, cu_q, cu_k, causal)
    assert o64.isnan().any() and (o64 == math.inf).any() and (o64 == -math.inf).any()
    same_kind(got, o64)
    ob, lb = ref.attend_bounds(o64.nan_to_num(0, 0, 0), mag.nan_to_num(0, 0, 0), reach, ends[-1], dim, dtype)
    within(got, o64, ob)
    seen = l64 > -math.inf
    assert torch.equal(lse.cpu()[~seen].double(), l64[~seen])
    assert ((lse.cpu().double() - l64).abs() <= lb)[seen].all()
