"""Refusals of the layer operators, on the host: the torch wrappers and the C
entry points reject bad arguments before anything is launched (no GPU needed)."""
import pytest
import torch

import gated_delta_rule_147_b200 as gdr
from gated_delta_rule_147_b200 import _layers, _lib, layers  # noqa: F401

P, N = 1 << 20, None  # a fake, aligned device address that no check follows
BAD, UNSUP, MIS = _lib.GDR_ERR_INVALID_ARG, _lib.GDR_ERR_UNSUPPORTED, _lib.GDR_ERR_MISALIGNED


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_wrappers_refuse_host_tensors_and_types():
    with pytest.raises(ValueError, match="CUDA tensors"):
        gdr.conv_fwd(t(1, 4, 8), t(8, 4))
    with pytest.raises(ValueError, match="CUDA tensors"):
        gdr.scan_step(t(1, 8), t(1, 8), t(8, 4), t(1, 1, 4), t(1, 1, 4), None, None, t(1, 8, 4))
    with pytest.raises(ValueError, match="CUDA tensors"):
        gdr.qk_norm_fwd(t(1, 4, 2, 8))
    with pytest.raises(TypeError, match="unsupported dtype"):
        gdr.conv_step(t(1, 8, dtype=torch.float16), t(8, 4), None, t(1, 3, 8))
    with pytest.raises(TypeError, match="unsupported dtype"):
        gdr.qk_norm_bwd(t(1, 4, 2, 8, dtype=torch.float64), dq=t(1, 4, 2, 8))


@pytest.mark.parametrize("bad,match", [
    (lambda: t(2, 5, 8), "shape"), (lambda: t(2, 4, 8, dtype=torch.float32), "dtype"),
    (lambda: t(2, 8, 4).transpose(1, 2), "innermost"),
    (lambda: t(2, 4, 1).expand(2, 4, 8), "innermost"),
])
def test_tensor_check(bad, match):
    with pytest.raises((TypeError, ValueError), match=match):
        _layers.check_tensor("x", bad(), (2, 4, 8), 1)


def test_tensor_check_takes_slices():
    x = t(2, 4, 24)[..., 8:16]
    assert _layers.check_tensor("x", x, (2, 4, 8), 1) == (96, 24, 1)
    m = t(2, 4, 20)[..., 4:12].view(2, 4, 2, 4)
    assert _layers.check_tensor("m", m, (2, 4, 2, 4), 2)[:2] == (80, 20)
    with pytest.raises(ValueError, match="last 2 axes"):
        _layers.check_tensor("m", t(2, 4, 2, 8)[..., :4], (2, 4, 2, 4), 2)


def test_results_stand_apart():
    a = t(4, 8)
    apart = _layers.check_apart
    apart("out", a[:2], "x", a[2:], False)
    apart("out", a[:2], "X0", None, False)
    apart("out", a[:2], "y", t(0, 8), False)
    with pytest.raises(ValueError, match="out overlaps x"):
        apart("out", a[:2], "x", a[1:], False)
    with pytest.raises(ValueError, match="overlaps"):  # a slice between the rows' other elements
        apart("out", a.view(-1)[4:8], "x", a[:, :4], False)
    apart("X_T", a, "X0", a, True)
    with pytest.raises(ValueError, match="overlaps"):  # the same start, not the same memory
        apart("X_T", a.view(-1)[:16], "X0", a[:, :4], True)


def conv(fn="fwd", **kw):
    a = dict(x=P, w=P, b=P, X0=P, len=N, dy=P, dXT=P, y=P, XT=P, dw=P, db=P, dX0=P, ws=P, nb=1 << 40, st=N, B=2, T=8,
             D=8, W=4, act=1, dt=0, wdt=0, gdt=0)
    a.update(kw)
    lib = _lib.load()
    if fn == "fwd":
        return lib.gdr_conv_fwd(a["x"], a["w"], a["b"], a["X0"], a["len"], a["y"], a["XT"], a["st"], a["B"], a["T"],
                                a["D"], a["W"], a["act"], a["dt"], a["wdt"], N)
    if fn == "step":
        return lib.gdr_conv_step(a["x"], a["w"], a["b"], a["X0"], a["y"], a["st"], a["B"], a["D"], a["W"], a["act"],
                                 a["dt"], a["wdt"], N)
    return lib.gdr_conv_bwd(a["x"], a["w"], a["b"], a["X0"], a["len"], a["dy"], a["dXT"], a["y"], a["dw"], a["db"],
                            a["dX0"], a["ws"], a["nb"], a["st"], a["B"], a["T"], a["D"], a["W"], a["act"], a["dt"],
                            a["wdt"], a["gdt"], N)


@pytest.mark.parametrize("fn", ["fwd", "bwd", "step"])
@pytest.mark.parametrize("kw,expect", [
    (dict(B=0), BAD), (dict(D=0), BAD), (dict(act=2), BAD), (dict(dt=5), BAD), (dict(w=N), BAD), (dict(x=N), BAD),
    (dict(W=1), UNSUP), (dict(W=5), UNSUP), (dict(dt=1, wdt=0, gdt=1), UNSUP), (dict(x=P + 1), MIS),
    (dict(w=P + 1), MIS),
])
def test_conv_rejects(fn, kw, expect):
    assert conv(fn, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(ws=N), BAD), (dict(nb=4), BAD), (dict(ws=P + 16), MIS), (dict(db=N), BAD), (dict(b=N), BAD),
    (dict(X0=N), BAD), (dict(dw=N), BAD), (dict(gdt=7), BAD), (dict(dt=1, wdt=1, gdt=0), UNSUP), (dict(dy=P + 1), MIS),
    (dict(T=-1), BAD),
])
def test_conv_bwd_rejects(kw, expect):
    assert conv("bwd", **kw) == expect


def scan(fn="fwd", **kw):
    a = dict(u=P, dl=P, A=P, Bm=P, Cm=P, D=P, z=P, bias=P, h0=P, len=N, y=P, hT=P, dy=P, du=P, ddl=P, dA=P, dB=P, dC=P,
             dD=P, dz=P, dbias=P, dh0=P, ws=P, nb=1 << 40, st=N, B=2, T=8, Dn=8, N=4, G=2, sp=1, dt=0, gdt=0)
    a.update(kw)
    lib = _lib.load()
    head = [a[k] for k in ("u", "dl", "A", "Bm", "Cm", "D", "z", "bias", "h0")]
    if fn == "fwd":
        return lib.gdr_scan_fwd(*head, a["len"], a["y"], a["hT"], a["ws"], a["nb"], a["st"], a["B"], a["T"], a["Dn"],
                                a["N"], a["G"], a["sp"], a["dt"], N)
    if fn == "step":
        return lib.gdr_scan_step(*head, a["y"], a["st"], a["B"], a["Dn"], a["N"], a["G"], a["sp"], a["dt"], N)
    return lib.gdr_scan_bwd(*head, a["len"], a["dy"], a["hT"], a["du"], a["ddl"], a["dA"], a["dB"], a["dC"], a["dD"],
                            a["dz"], a["dbias"], a["dh0"], a["ws"], a["nb"], a["st"], a["B"], a["T"], a["Dn"], a["N"],
                            a["G"], a["sp"], a["dt"], a["gdt"], N)


@pytest.mark.parametrize("fn", ["fwd", "bwd", "step"])
@pytest.mark.parametrize("kw,expect", [
    (dict(B=0), BAD), (dict(Dn=0), BAD), (dict(N=0), BAD), (dict(G=3), BAD), (dict(G=0), BAD), (dict(dt=2), BAD),
    (dict(A=N), BAD), (dict(u=N), BAD), (dict(Bm=N), BAD), (dict(N=129), UNSUP), (dict(dl=P + 1), MIS),
    (dict(A=P + 2), MIS),
])
def test_scan_rejects(fn, kw, expect):
    assert scan(fn, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(ws=N), BAD), (dict(nb=64), BAD), (dict(ws=P + 16), MIS), (dict(dD=N), BAD), (dict(dz=N), BAD),
    (dict(dbias=N), BAD), (dict(h0=N), BAD), (dict(dA=N), BAD), (dict(dy=N), BAD), (dict(gdt=3), BAD),
    (dict(dt=1, gdt=0), UNSUP), (dict(dy=P + 1), MIS), (dict(T=-1), BAD),
])
def test_scan_bwd_rejects(kw, expect):
    assert scan("bwd", **kw) == expect


def norm(fn="fwd", **kw):
    a = dict(q=P, k=P, qw=P, kw=P, pos=P, f=P, gq=P, gk=P, qo=P, ko=P, dqw=P, dkw=P, ws=P, nb=1 << 40, st=N, B=2, T=4,
             Hq=4, Hk=2, d=64, rot=32, kind=1, lay=0, eps=1e-6, qs=1.0, rs=1.0, p64=0, dt=0, wdt=0, gdt=0)
    a.update(kw)
    lib = _lib.load()
    head = [a[k] for k in ("q", "k", "qw", "kw", "pos", "f")]
    tail = [a[k] for k in ("B", "T", "Hq", "Hk", "d", "rot", "kind", "lay", "eps", "qs", "rs", "p64", "dt", "wdt")]
    if fn == "fwd":
        return lib.gdr_qk_norm_fwd(*head, a["qo"], a["ko"], a["st"], *tail, N)
    return lib.gdr_qk_norm_bwd(*head, a["gq"], a["gk"], a["qo"], a["ko"], a["dqw"], a["dkw"], a["ws"], a["nb"],
                               a["st"], *tail, a["gdt"], N)


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,expect", [
    (dict(B=0), BAD), (dict(Hq=0), BAD), (dict(d=0), BAD), (dict(rot=31), BAD), (dict(rot=66), BAD), (dict(f=N), BAD),
    (dict(rot=0), BAD), (dict(kind=0), BAD), (dict(kind=4), BAD), (dict(lay=2), BAD), (dict(eps=0.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(k=N), BAD), (dict(Hk=0), BAD), (dict(q=N), BAD), (dict(p64=2), BAD),
    (dict(d=257), UNSUP), (dict(dt=1, wdt=0, gdt=1), UNSUP), (dict(q=P + 1), MIS), (dict(pos=P + 4, p64=1), MIS),
])
def test_norm_rejects(fn, kw, expect):
    assert norm(fn, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(ws=N), BAD), (dict(nb=64), BAD), (dict(ws=P + 16), MIS), (dict(dqw=N), BAD), (dict(gq=N), BAD),
    (dict(gdt=2), BAD), (dict(qo=P + 2), MIS),
])
def test_norm_bwd_rejects(kw, expect):
    assert norm("bwd", **kw) == expect


def test_workspace_sizes():
    # conv: (W + 1) sums per channel for each chunk of tokens of each sequence
    assert _lib.gdr_conv_bwd_workspace_size(1, 0, 8, 4) == 256
    assert _lib.gdr_conv_bwd_workspace_size(2, 16, 512, 4) == 2 * 5 * 512 * 4
    assert _lib.gdr_conv_bwd_workspace_size(2, 16, 512, 5) == 0
    # scan: 32 channels x 16 states every 8 tokens; dB and dC of the one tile; parameters
    assert _lib.gdr_scan_bwd_workspace_size(1, 20, 16, 16, 1) == 3 * 2048 + 20 * 32 * 4 + 1280
    # the same split in two chunks, with the maps of each (decay and end, twice)
    assert _lib.gdr_scan_bwd_workspace_size(1, 512, 16, 16, 1) == 64 * 2048 + 512 * 32 * 4 + 2304 + 2 * 2 * 4096
    assert _lib.gdr_scan_fwd_workspace_size(1, 767, 16, 16, 1) == 0  # two chunks of 256 do not pay
    assert _lib.gdr_scan_fwd_workspace_size(1, 768, 16, 16, 1) == 3 * 8192
    assert _lib.gdr_scan_fwd_workspace_size(4, 4096, 4096, 16, 1) == 0
    assert _lib.gdr_scan_fwd_workspace_size(1, 768, 16, 129, 1) == 0
    assert _lib.gdr_scan_bwd_workspace_size(1, 20, 16, 16, 3) == 0
    assert _lib.gdr_qk_norm_bwd_workspace_size(0) == 0
