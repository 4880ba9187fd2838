"""A torch binding that cannot be built costs its own compilation and no more:
libfd.so is not compiled again for it, and no older binding stays in use."""
import os

import pytest

from split_kv_decode_paged_gb300 import build as B


@pytest.fixture
def place(fdlib, tmp_path, monkeypatch):
    """A current libfd.so (an empty file) and no compilers."""
    lib, binding, calls = tmp_path / "libfd.so", tmp_path / "_fd_torch.so", []
    lib.write_bytes(b"")
    monkeypatch.setattr(B, "LIB", str(lib))
    monkeypatch.setattr(B, "BINDING", str(binding))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "obj"))

    def no(*a, **kw):
        calls.append("nvcc")
        raise RuntimeError("no nvcc")

    def failing():
        calls.append("binding")
        raise RuntimeError("no g++")
    monkeypatch.setattr(B, "nvcc", no)
    monkeypatch.setattr(B, "build_binding", failing)
    return lib, binding, calls


def test_missing_binding_is_built_alone(place, capsys):
    lib, binding, calls = place
    assert B.build() == str(lib) and B.build() == str(lib)
    assert calls == ["binding", "binding"] and "no native torch binding" in capsys.readouterr().err


def test_an_older_binding_does_not_stay(place):
    lib, binding, calls = place
    binding.write_bytes(b"")
    os.utime(binding, (1, 1))
    B.build()
    assert calls == ["binding"] and not binding.exists()


def test_nothing_is_built_twice(place):
    lib, binding, calls = place
    binding.write_bytes(b"")
    assert B.build() == str(lib) and not calls


def test_an_older_library_is_compiled(place):
    lib, binding, calls = place
    binding.write_bytes(b"")
    os.utime(lib, (1, 1))
    with pytest.raises(RuntimeError, match="no nvcc"):
        B.build()
    assert calls == ["nvcc"]
