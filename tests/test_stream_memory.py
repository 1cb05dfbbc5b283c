"""CPU test of where the binding takes a call's memory from: with a stream given, every output and
scratch tensor is allocated while that stream is the current one (the allocator hands a block out in
the order of one stream only), and outputs are recorded on the caller's current stream."""
import contextlib

import pytest

from gemm_qmm_nbits_amd import qmm as Q


class FakeTensor:
    def __init__(self, stream):
        self.made_on, self.recorded = stream, []

    def record_stream(self, stream):
        self.recorded.append(stream)


class FakeTorch:
    uint8 = "uint8"

    def __init__(self):
        self.now, self.cuda = "current", self

    @contextlib.contextmanager
    def stream(self, s):
        before, self.now = self.now, s
        yield
        self.now = before

    def current_stream(self, device=None):
        return self.now

    def empty(self, shape, dtype=None, device=None):
        return FakeTensor(self.now)

    zeros = empty


class Like:
    device = "cuda:0"


@pytest.fixture
def fake(monkeypatch):
    t = FakeTorch()
    monkeypatch.setattr(Q, "_torch", lambda: t)
    return t


def test_outputs(fake):
    t = Q._new((2, 3), "f32", Like, "side")
    assert t.made_on == "side" and t.recorded == ["current"]
    t = Q._new((2, 3), "f32", Like, None)
    assert t.made_on == "current" and not t.recorded


@pytest.mark.parametrize("zeroed", [False, True])
def test_scratch(fake, zeroed):
    assert Q._temporary(64, Like, "side", zeroed=zeroed).made_on == "side"
    assert Q._temporary(64, Like, None, zeroed=zeroed).made_on == "current"


def test_no_entry_allocates_by_itself():
    """Every entry that takes a stream takes its memory from these two."""
    import inspect

    for name, f in inspect.getmembers(Q, inspect.isfunction):
        if "stream" in inspect.signature(f).parameters and name not in ("_new", "_temporary"):
            text = inspect.getsource(f).replace("torch.empty(0, dtype=out_dtype)", "")
            assert "torch.empty" not in text and "torch.zeros" not in text, name
