"""The native binding (built with g++ against Python's and torch's headers) is
needed by the calls that go through it alone: where it cannot be built, the
library and its other calls work as they are."""
import pytest
import torch

from moe_matvec_gb300 import api


@pytest.fixture
def unbuildable(monkeypatch):
    def fail(*a, **k):
        raise RuntimeError("no headers here")
    monkeypatch.setattr(api._build, "build_binding", fail)
    monkeypatch.setattr(api, "_lib", None)
    monkeypatch.setattr(api, "_native", None)


def test_the_library_loads_without_the_binding(unbuildable):
    lib = api.load()
    assert lib.qmv_row_bytes(api.Q8_0, 256) == 272
    assert lib.qmv_run(99, None, None, None, 1, 256, 1, None) == -1  # refused by the library itself
    with api.using(lib):
        assert api.kv_page_bytes(128, 64) == 16 + 2 * 64 * 128


def test_calls_through_the_binding_say_why(unbuildable):
    x = torch.zeros(2, 512)
    with pytest.raises(RuntimeError, match="no headers here"):
        api.rms_norm(x, torch.ones(512))


def test_the_binding_follows_the_active_library(monkeypatch):
    seen = []
    monkeypatch.setattr(api, "_native", None)
    native = api._nat()

    class Spy:
        def bind(self, *a):
            seen.append(a)
            native.bind(*a)

    monkeypatch.setattr(api, "_native", Spy())
    with api.using(api.load()):
        pass
    assert len(seen) == 2 and seen[0] == seen[1] and len(seen[0]) == 9
