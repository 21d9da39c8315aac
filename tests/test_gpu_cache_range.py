"""The ends of what comes back finite from a microscaled cache, and through the attention over it."""
import math

import pytest
import torch

import varlen_top_select_amd as vts

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16

# the largest power of two, the least value that rounds to twice that, and what those below give
ENDS = [(F16, 4, 2.0 ** 15, 1.75, 1.5), (F16, 8, 2.0 ** 15, 1.9375, 1.875), (BF16, 4, 2.0 ** 127, 1.75, 1.5),
        (BF16, 8, 2.0 ** 127, 1.9375, 1.875)]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype,bits,power,up,down", ENDS)
def test_values_next_to_the_largest(dtype, bits, power, up, down, sign):
    """A block's largest value from up * power on is an infinity, one below is down * power."""
    caches = [torch.zeros(1, 16, 1, 8 * bits, dtype=torch.uint8, device=DEV) for _ in "kv"]
    scales = [torch.zeros(1, 16, 1, 2, dtype=torch.uint8, device=DEV) for _ in "kv"]
    least = torch.tensor(up * power, dtype=dtype)
    assert float(least) == up * power
    below = (least.view(torch.int16) - 1).view(dtype)
    x = torch.zeros(2, 1, 64, dtype=dtype)
    x[0, 0, 5], x[1, 0, 5] = sign * below, sign * least
    x[:, 0, 40] = 1
    x = x.to(DEV)
    slots = torch.arange(2, dtype=torch.int32, device=DEV)
    kw = dict(k_scales=scales[0], v_scales=scales[1])
    vts.write_cache(x, x, x, slots, *caches, **kw)
    for got in vts.read_cache(*caches, slots, dtype=dtype, **kw):
        assert float(got[0, 0, 5]) == sign * down * power
        assert float(got[1, 0, 5]) == sign * math.inf
        assert (got[:, 0, 40] == 1).all()
    q = torch.zeros(2, 1, 1, 64, dtype=dtype, device=DEV)
    q[..., 40] = 1
    table = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    out, _ = vts.tree_attention(q, *caches, table, torch.tensor([1, 1], dtype=torch.int32, device=DEV),
                                slots=slots.view(2, 1), **kw)
    assert float(out[0, 0, 0, 5]) == sign * down * power and float(out[0, 0, 0, 40]) == 1
