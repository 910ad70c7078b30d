"""When the build compiles again. CPU only; nothing is compiled for the test's own versions."""
import importlib.metadata

import pytest

from exact_io_aware_13_gb300 import build as libbuild


@pytest.fixture
def compiled(monkeypatch):
    """What build() compiles from here on, by name."""
    libbuild.build()
    calls = []
    monkeypatch.setattr(libbuild, "_compile", lambda src, *a: calls.append(src) or src)
    monkeypatch.setattr(libbuild, "_compile_binding", lambda *a: calls.append("binding") or "binding.o")
    monkeypatch.setattr(libbuild, "_link_binding", lambda obj: calls.append("link"))
    return calls


def test_nothing_new(compiled):
    libbuild.build()
    assert compiled == []


def test_another_torch_rebuilds_the_binding_alone(compiled, monkeypatch):
    """_binding.so holds torch's C++ interface: newer than every source, it is still another
    version's."""
    real = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0" if name == "torch" else real(name))
    libbuild.build()
    assert compiled == ["binding", "link"]
