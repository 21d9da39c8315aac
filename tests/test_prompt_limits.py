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
