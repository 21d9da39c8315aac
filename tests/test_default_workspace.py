"""The default workspace of a stream outlives its replacement by a larger one: a
graph captured with it keeps its address.  On the CPU with a stand-in for the
library; the replays themselves are in tests/test_gpu_default_workspace.py."""
import weakref

import pytest
import torch

import varlen_top_select_amd as vts


class Library:
    @staticmethod
    def vts_workspace_init(ptr, nbytes, stream):
        return 0


@pytest.fixture
def cpu(monkeypatch):
    monkeypatch.setattr(vts, "_WS_CACHE", {})
    monkeypatch.setattr(vts, "library", lambda: Library)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return torch.device("cpu")


@pytest.mark.parametrize("kind", ["select", "decode"])
def test_a_replaced_workspace_stays(cpu, kind):
    small = vts._default_workspace(1000, cpu, 0, kind)
    at, alive = small.data_ptr(), weakref.ref(small)
    del small
    large = vts._default_workspace(5000, cpu, 0, kind)
    assert large.data_ptr() != at and large.numel() >= 5000
    assert alive() is not None, "its memory is free for others"
    assert vts._default_workspace(5000, cpu, 0, kind) is large
    assert vts._default_workspace(10, cpu, 0, kind) is large


def test_replaced_workspaces_are_few(cpu, monkeypatch):
    """A shape that grows bit by bit: what is kept holds less than the last one."""
    kept = []
    monkeypatch.setattr(vts, "_WS_REPLACED", kept, raising=False)
    for need in range(1000, 100000, 777):
        ws = vts._default_workspace(need, cpu, 0)
        assert ws.numel() >= need
    assert 0 < len(kept) < 8 and sum(x.numel() for x in kept) < ws.numel() < 200000


def test_streams_and_kinds_have_their_own(cpu):
    got = [vts._default_workspace(100, cpu, s, kind) for s in (0, 7) for kind in ("select", "decode")]
    assert len({x.data_ptr() for x in got}) == 4
