"""Ends of what vts_prompt_attention takes, on the host alone: batches of no sequence, and the
largest grid."""
import pytest

from tests.test_cache_host import A, HIP, NO_GPU, OK, UNSUPPORTED, lib, prompts  # noqa: F401


def call(lib, clear, **kw):  # noqa: F811
    return lib.vts_prompt_attention(prompts(**kw), 1, 0.1, 1 << 40, None, clear, None, 0, None)


@pytest.mark.parametrize("kw", [dict(tq=1), dict(tq=31), dict(tq=100, heads=8), dict(tq=5000), dict(cu_q=None, cu_k=None)])
def test_no_sequence(lib, kw):  # noqa: F811
    """A batch of none leaves all rows as they are: nothing is started, be there a tile's rows or fewer."""
    assert call(lib, 0, batch=0, **kw) == OK


@pytest.mark.skipif(not NO_GPU, reason="pointers to nothing")
@pytest.mark.parametrize("over", [0, 1])
def test_the_largest_grid(lib, over):  # noqa: F811
    """tiles * kv_heads below 2^24 - 64: with the 64 workgroups for rows of no sequence a grid of 256
    threads each stays below 2^32."""
    batch = 2 ** 23 - 65 + over  # and 2^23 full tiles of 128 rows
    got = call(lib, 1, heads=1, kv=1, qs=(128, 128), ks=(128, 128), vs=(128, 128), tq=2 ** 30, tk=100, batch=batch)
    if over:
        assert got == UNSUPPORTED
    else:  # (as far as the device, which is not there)
        assert got == HIP
