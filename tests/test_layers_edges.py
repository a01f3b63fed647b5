"""The layer operators' host side at the ends of what they take (no GPU needed)."""
import pytest
import torch

from gated_delta_rule_147_b200 import _lib, build, layers  # noqa: F401
from gated_delta_rule_147_b200 import _layers

P = 1 << 20  # a fake, aligned device address that no check follows


def test_a_result_in_place_has_its_inputs_layout():
    """The same bytes in another order are not the same rows."""
    buf = torch.zeros(2, 3, 4, 8)
    apart = _layers.check_apart
    apart("q_out", buf, "q", buf, True)
    apart("q_out", buf.view(6, 1, 4, 8), "q", buf, True)
    with pytest.raises(ValueError, match="q_out overlaps q"):
        apart("q_out", buf.view(2, 4, 3, 8), "q", buf.transpose(1, 2), True)
    with pytest.raises(ValueError, match="q_out overlaps q"):
        apart("q_out", buf, "q", buf[:, :, :, :1].expand(2, 3, 4, 8), True)
    one = torch.zeros(2, 1, 4, 8)  # an axis of one has no order
    apart("q_out", one.view(2, 4, 1, 8), "q", one.transpose(1, 2), True)


def commands_of_a_build(monkeypatch, tmp_path):
    got = []
    monkeypatch.setattr(build, "OBJDIR", str(tmp_path / "obj"))
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: got.append(list(cmd)))
    assert build.build(force=True) == build.LIB
    return got


def test_the_library_builds_without_torch(monkeypatch, tmp_path):
    """C callers need nvcc alone: no torch, then no Python module, but the library."""
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    got = commands_of_a_build(monkeypatch, tmp_path)
    assert not any(build.BINDING in " ".join(c) or build.MODULE in c for c in got)
    assert sum(c[-1].endswith(".cu") for c in got) == len(build.SOURCES) and build.LIB in got[-1]
    monkeypatch.setattr(build, "MODULE", str(tmp_path / "none.so"))  # its absence does not call for a build
    monkeypatch.setattr(build.os.path, "getmtime", lambda f: 1.0)
    assert not build._stale()


def test_the_module_builds_with_the_headers_of_the_nvcc_in_use(monkeypatch, tmp_path):
    nvcc = tmp_path / "cuda" / "bin" / "nvcc"
    nvcc.parent.mkdir(parents=True)
    nvcc.write_text("")
    monkeypatch.setenv("NVCC", str(nvcc))
    got = commands_of_a_build(monkeypatch, tmp_path)
    binding = next(c for c in got if c[-1].endswith(build.BINDING))
    assert str(tmp_path / "cuda" / "include") in binding and "/usr/local/cuda/include" not in binding
    assert build.MODULE in got[-1]


def test_workspace_sizes_are_declared_as_sizes():
    """ctypes takes a C int unless told otherwise, which cuts a size to 32 bits."""
    lib = _lib.load()
    for name in _lib.EXPORTS:
        if name.endswith(("_workspace_size", "_capacity")):
            assert getattr(lib, name).restype is _lib.ctypes.c_size_t, name
            assert getattr(lib, name).argtypes is not None, name
