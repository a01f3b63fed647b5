"""The 64-bit forms that the layer operators are tested against: their
gradients agree with automatic differentiation and with differences."""
import pytest
import torch

import layers_ref as R


def rnd(*s, seed=[0]):
    seed[0] += 1
    return torch.randn(s, dtype=torch.float64, generator=torch.Generator().manual_seed(seed[0]))


def agree(got, want, what):
    assert torch.allclose(got, want, rtol=1e-9, atol=1e-11), (what, (got - want).abs().max())


def differences(f, x, got, what):
    """A directional central difference of the scalar f at x against the gradient."""
    d = rnd(*x.shape)
    h = 1e-6
    num = (f(x + h * d) - f(x - h * d)) / (2 * h)
    assert abs(num - (got * d).sum()) <= 1e-7 * (1 + abs(num)), what


@pytest.mark.parametrize("act", [True, False])
def test_conv(act):
    x, w, b, X0, dy, dX = rnd(2, 6, 3), rnd(3, 4), rnd(3), rnd(2, 3, 3), rnd(2, 6, 3), rnd(2, 3, 3)
    lengths = [6, 2]
    leaves = {"dx": x, "dweight": w, "dbias": b, "dX0": X0}
    for t in leaves.values():
        t.requires_grad_()

    def loss(x, w, b, X0):
        tot = 0
        for i, n in enumerate(lengths):
            rows = torch.cat([X0[i], x[i, :n]])
            p = torch.nn.functional.conv1d(rows.T[None], w[:, None], b, groups=3)[0].T
            y = torch.nn.functional.silu(p) if act else p
            tot = tot + (y * dy[i, :n]).sum() + (rows[n:] * dX[i]).sum()
        return tot
    grads = torch.autograd.grad(loss(x, w, b, X0), list(leaves.values()))
    v, m = R.conv(x, w, b, X0, lengths, act, dy, dX)
    for (k, _), g in zip(leaves.items(), grads):
        agree(v[k], g, k)
        assert (m[k] >= v[k].abs() - 1e-12).all(), k
    with torch.no_grad():
        differences(lambda t: loss(t, w, b, X0), x, v["dx"], "dx")


def scan_loss(u, dl, A, Bm, Cm, D, z, h0, bias, dy, dh, softplus, lengths):
    tot, K = 0, u.shape[2] // Bm.shape[2]
    for b, n in enumerate(lengths):
        h = h0[b]
        for t in range(n):
            raw = dl[b, t] + bias
            dt = torch.nn.functional.softplus(raw) if softplus else raw
            h = torch.exp(dt[:, None] * A) * h + (dt * u[b, t])[:, None] * Bm[b, t].repeat_interleave(K, 0)
            y = (Cm[b, t].repeat_interleave(K, 0) * h).sum(1) + D * u[b, t]
            tot = tot + (y * torch.nn.functional.silu(z[b, t]) * dy[b, t]).sum()
        tot = tot + (h * dh[b]).sum()
    return tot


@pytest.mark.parametrize("softplus", [True, False])
def test_scan(softplus):
    B, T, D, N, G = 2, 5, 4, 3, 2
    a = [rnd(B, T, D), 0.3 * rnd(B, T, D), -rnd(D, N).abs(), rnd(B, T, G, N), rnd(B, T, G, N), rnd(D), rnd(B, T, D),
         rnd(B, D, N), rnd(D)]
    dy, dh = rnd(B, T, D), rnd(B, D, N)
    names = ["du", "ddelta", "dA", "dB", "dC", "dD", "dz", "dh0", "ddelta_bias"]
    for t in a:
        t.requires_grad_()
    lengths = [5, 3]
    grads = torch.autograd.grad(scan_loss(*a, dy, dh, softplus, lengths), a)
    v, m, e = R.scan(*a, softplus, lengths, dy, dh)
    for k, g in zip(names, grads):
        agree(v[k], g, k)
        assert (m[k] >= v[k].abs() - 1e-12).all(), k
        assert (e[k] >= m[k] * (1 - 1e-9)).all() or k == "dD", k
    with torch.no_grad():
        for i, k in enumerate(names):
            differences(lambda t: scan_loss(*a[:i], t, *a[i + 1:], dy, dh, softplus, lengths), a[i], v[k], k)


@pytest.mark.parametrize("kind,layout", [("l2", "half"), ("rms", "interleaved")])
def test_norm(kind, layout):
    x, w, dout = rnd(2, 3, 2, 8), rnd(8) if kind == "rms" else None, rnd(2, 3, 2, 8)
    f = torch.tensor([1.0, 0.1, 0.01], dtype=torch.float64)
    x.requires_grad_()

    def loss(x):
        n = x / x.norm(dim=-1, keepdim=True) if kind == "l2" else \
            x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        ang = torch.arange(3.0, dtype=torch.float64)[:, None, None] * f
        unit = torch.polar(torch.ones_like(ang), ang)
        if layout == "half":
            y = torch.complex(n[..., :3], n[..., 3:6]) * unit
            y = torch.cat([y.real, y.imag], -1)
        else:
            y = torch.view_as_real(torch.view_as_complex(n[..., :6].reshape(2, 3, 2, 3, 2)) * unit).flatten(-2)
        return (torch.cat([1.5 * y, n[..., 6:]], -1) * dout * 0.7).sum()
    g, = torch.autograd.grad(loss(x), x)
    v, m = R.norm(x, w, kind, scale=0.7, inv_freq=f, layout=layout, rscale=1.5, dout=dout)
    agree(v["dx"], g, "dx")
    assert (m["dx"] >= v["dx"].abs() - 1e-12).all()
    with torch.no_grad():
        differences(loss, x, v["dx"], "dx")
