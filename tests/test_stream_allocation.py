"""What a call allocates comes from the pool of the stream it runs on (host only, a stand-in for torch)."""
import contextlib
import types

import pytest

import selective_scan_segmented_amd as sfm


class FakeTorch:
    """Streams are strings; a tensor knows whose pool it came from and which other streams hold it."""

    def __init__(self):
        self.now = "current"

    def empty(self, shape, dtype=None, device=None):
        t = types.SimpleNamespace(shape=shape, dtype=dtype, device=device, pool=self.now, held=[])
        t.record_stream = t.held.append
        return t

    def empty_like(self, t):
        return self.empty(t.shape, t.dtype, t.device)

    @property
    def cuda(self):
        return types.SimpleNamespace(stream=self.stream, current_stream=lambda device=None: self.now)

    @contextlib.contextmanager
    def stream(self, s):
        before, self.now = self.now, s
        yield
        self.now = before


@pytest.fixture
def fake(monkeypatch):
    t = FakeTorch()
    monkeypatch.setattr(sfm, "_torch_module", t)
    return t


@pytest.mark.parametrize("like", [False, True])
def test_a_stream_of_the_caller(fake, like):
    src = fake.empty((2, 3), "f32", "gpu")
    t = sfm._new_like(src, "side") if like else sfm._new((2, 3), "f32", "gpu", "side")
    assert t.pool == "side" and (t.shape, t.dtype, t.device) == ((2, 3), "f32", "gpu")
    assert "current" in t.held  # the caller has it there
    assert fake.now == "current"


@pytest.mark.parametrize("like", [False, True])
def test_the_current_stream(fake, like):
    src = fake.empty((2, 3), "f32", "gpu")
    t = sfm._new_like(src, None) if like else sfm._new((2, 3), "f32", "gpu", None)
    assert t.pool == "current" and not t.held


def test_a_workspace_is_its_streams_alone(fake):
    """Nobody has it on the current stream, so its memory is there for the next call as soon as the call returns."""
    fake.uint8 = "uint8"
    t = sfm._scratch(64, "gpu", "side")
    assert t.pool == "side" and not t.held and (t.shape, t.dtype, t.device) == (64, "uint8", "gpu")
    assert sfm._scratch(64, "gpu", None).pool == "current"
