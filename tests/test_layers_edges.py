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


LONGEST = 2 ** 31 - 1 - 4096


def entry(fn, **kw):
    """Status of one entry point, with fake pointers and dense arrays."""
    a = dict(B=1, T=1, D=1, W=2, N=1, G=1, H=1, Hk=1, d=1)
    a.update(kw)
    lib, n = _lib.load(), None
    B, T, D, W, N, G, H, Hk, d = (a[k] for k in ("B", "T", "D", "W", "N", "G", "H", "Hk", "d"))
    if fn == "conv_fwd":
        return lib.gdr_conv_fwd(P, P, n, n, n, P, n, n, B, T, D, W, 0, 0, 0, n)
    if fn == "conv_bwd":
        return lib.gdr_conv_bwd(P, P, n, n, n, P, n, P, P, n, n, P, 1 << 50, n, B, T, D, W, 0, 0, 0, 0, n)
    if fn == "conv_step":
        return lib.gdr_conv_step(P, P, n, P, P, n, B, D, W, 0, 0, 0, n)
    if fn == "scan_fwd":
        return lib.gdr_scan_fwd(P, P, P, P, P, n, n, n, n, n, P, n, n, 0, n, B, T, D, N, G, 0, 0, n)
    if fn == "scan_bwd":
        return lib.gdr_scan_bwd(P, P, P, P, P, n, n, n, n, n, P, n, P, P, P, P, P, n, n, n, n, P, 1 << 50, n, B, T, D, N, G,
                                0, 0, 0, n)
    if fn == "scan_step":
        return lib.gdr_scan_step(P, P, P, P, P, n, n, n, P, P, n, B, D, N, G, 0, 0, n)
    if fn == "qk_norm_fwd":
        return lib.gdr_qk_norm_fwd(P, P, n, n, n, n, P, P, n, B, T, H, Hk, d, 0, 0, 0, 1e-6, 1.0, 1.0, 0, 0, 0, n)
    return lib.gdr_qk_norm_bwd(P, P, n, n, n, n, P, P, P, P, n, n, n, 0, n, B, T, H, Hk, d, 0, 0, 0, 1e-6, 1.0, 1.0, 0, 0, 0,
                               0, n)


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: for hosts without a GPU")
@pytest.mark.parametrize("fn,axes", [("conv_fwd", "BTD"), ("conv_bwd", "BTD"), ("conv_step", "BD"), ("scan_fwd", "BTD"),
                                     ("scan_bwd", "BTD"), ("scan_step", "BD"), ("qk_norm_fwd", "H"), ("qk_norm_bwd", "H")])
def test_axes_that_the_kernels_would_count_past_are_refused(fn, axes):
    """Chunks, steps and vectors are rounded up and counted in int."""
    for ax in axes:
        for size in (2 ** 31 - 1, LONGEST + 1):
            assert entry(fn, **{ax: size}) == _lib.GDR_ERR_UNSUPPORTED, (ax, size)
    if fn.startswith("qk_norm"):
        assert entry(fn, H=2 ** 30, Hk=2 ** 30) == _lib.GDR_ERR_UNSUPPORTED
    sizes = {"conv_bwd": lambda T: _lib.gdr_conv_bwd_workspace_size(1, T, 1, 2),
             "scan_fwd": lambda T: _lib.gdr_scan_fwd_workspace_size(1, T, 1, 1, 1),
             "scan_bwd": lambda T: _lib.gdr_scan_bwd_workspace_size(1, T, 1, 1, 1)}
    if fn in sizes:
        assert sizes[fn](LONGEST + 1) == 0 and sizes[fn](LONGEST) > 0
