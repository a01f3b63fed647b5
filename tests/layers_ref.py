"""64-bit CPU forms of the layer operators, token by token, for the tests.

Every function also gives, for each result, the magnitude its rounding errors
scale with: the same sums over absolute values. A test's tolerance is then
  half a step of the output type x |result|  +  K 2^-24 x magnitude,
K the number of fp32 roundings on the longest path into the result.
"""
import torch

U32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, ref, mag, k, what):
    """got (any dtype, any device) against the 64-bit ref within the derived bound."""
    got64 = got.detach().double().cpu()
    assert got64.shape == ref.shape, (what, got64.shape, ref.shape)
    assert torch.isfinite(got64).all(), f"{what}: non-finite values"
    tol = half_step(got.dtype) * ref.abs() + k * U32 * (1 + half_step(got.dtype)) * mag + 1e-37
    over = ((got64 - ref).abs() / tol).max().item() if ref.numel() else 0.0
    assert over <= 1.0, f"{what}: error is {over:.3g} times the bound"


def f64(t):
    return None if t is None else t.detach().double().cpu()


def lens(lengths, B, T):
    if lengths is None:
        return [T] * B
    return [min(max(int(n), 0), T) for n in lengths]


def silu(p):
    s = torch.special.expit(p)
    return p * s, s * (1 + p * (1 - s))


# |silu'| <= 1.1, |silu''| <= 0.5 everywhere

def conv(x, w, bias=None, X0=None, lengths=None, act=True, dy=None, dX_T=None):
    """Returns ({name: value}, {name: magnitude})."""
    x, w, bias, X0, dy, dX_T = map(f64, (x, w, bias, X0, dy, dX_T))
    B, T, D = x.shape
    W = w.shape[1]
    z = lambda *s: torch.zeros(s, dtype=torch.float64)  # noqa: E731
    v = {"y": z(B, T, D), "X_T": z(B, W - 1, D), "dx": z(B, T, D), "dX0": z(B, W - 1, D), "dweight": z(D, W),
         "dbias": z(D)}
    m = {k: t.clone() for k, t in v.items()}
    for b, n in enumerate(lens(lengths, B, T)):
        rows = torch.cat([X0[b] if X0 is not None else z(W - 1, D), x[b, :n]])
        v["X_T"][b] = rows[n:n + W - 1]
        dr, mr = z(n + W - 1, D), z(n + W - 1, D)
        if dX_T is not None:
            dr[n:] += dX_T[b]
            mr[n:] += dX_T[b].abs()
        for t in range(n):
            win = rows[t:t + W]
            p = (w.T * win).sum(0) + (0 if bias is None else bias)
            pm = (w.T * win).abs().sum(0) + (0 if bias is None else bias.abs())
            f, df = silu(p) if act else (p, torch.ones_like(p))
            v["y"][b, t], m["y"][b, t] = f, 1.1 * pm
            if dy is None:
                continue
            dp, dm = dy[b, t] * df, dy[b, t].abs() * ((1.1 + 0.5 * pm) if act else 1.0)
            dr[t:t + W] += w.T * dp
            mr[t:t + W] += w.T.abs() * dm
            v["dweight"] += (dp * win).T
            m["dweight"] += (dm * win.abs()).T
            v["dbias"] += dp
            m["dbias"] += dm
        v["dX0"][b], v["dx"][b, :n] = dr[:W - 1], dr[W - 1:]
        m["dX0"][b], m["dx"][b, :n] = mr[:W - 1], mr[W - 1:]
    return v, m


def scan(u, delta, A, Bm, Cm, D=None, z=None, h0=None, bias=None, softplus=False, lengths=None, dy=None, dh_T=None):
    """Values of the forward (y, h_T) and, with dy, of every gradient; their
    magnitudes; and bounds on the error of a fp32 evaluation in units of U32,
    carried through the recurrence. The bounds count, per operation:
      dt    10 + 3 |raw| relative (sum, exponential with a rounded argument, quotient, series)
      a     |dt A| times dt's and 3 more (A log2 e, the product, its rounding), and 6
            (4 of the exponential, one each of the running product and the sum)
      silu  12 + 2 |z|, its derivative 12 + 2 |z| of 1.1
      a sum of n products: n + 1."""
    u, delta, A, Bm, Cm, D, z, h0, bias, dy, dh_T = map(f64, (u, delta, A, Bm, Cm, D, z, h0, bias, dy, dh_T))
    Bn, T, Dn = u.shape
    G, N = Bm.shape[2:]
    K = Dn // G
    zero = lambda *s: torch.zeros(s, dtype=torch.float64)  # noqa: E731
    wide = lambda t: t.repeat_interleave(K, 0)  # noqa: E731  [G, N] -> [D, N]
    fold = lambda t: t.view(G, K, N).sum(1)  # noqa: E731
    names = {"y": (Bn, T, Dn), "h_T": (Bn, Dn, N), "du": (Bn, T, Dn), "ddelta": (Bn, T, Dn), "dz": (Bn, T, Dn),
             "dB": (Bn, T, G, N), "dC": (Bn, T, G, N), "dA": (Dn, N), "dD": (Dn,), "ddelta_bias": (Dn,),
             "dh0": (Bn, Dn, N)}
    v = {k: zero(*s) for k, s in names.items()}
    m = {k: zero(*s) for k, s in names.items()}
    e = {k: zero(*s) for k, s in names.items()}
    skip = zero(Dn) if D is None else D
    for b, n in enumerate(lens(lengths, Bn, T)):
        h = zero(Dn, N) if h0 is None else h0[b].clone()
        H, Eh = h.abs(), zero(Dn, N)
        tape = []
        for t in range(n):
            ut, raw = u[b, t], delta[b, t] + (0 if bias is None else bias)
            dt = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
            edt = 10 + 3 * raw.abs() if softplus else 1.0 + 0 * raw  # relative
            if bias is not None and not softplus:
                edt = 1 + (delta[b, t].abs() + bias.abs()) / raw.abs().clamp(min=1e-30)
            x = dt[:, None] * A
            a = torch.exp(x)
            ea = x.abs() * (edt[:, None] + 3) + 6  # relative
            Bx, Cx = wide(Bm[b, t]), wide(Cm[b, t])
            hp, Hp, Ep = h, H, Eh
            inp = (dt * ut)[:, None] * Bx
            h = a * h + inp
            H = a * H + inp.abs()
            Eh = a * Ep + a * ea * Hp + inp.abs() * (edt[:, None] + 3) + H
            yh = (Cx * h).sum(1) + skip * ut
            Yh = (Cx.abs() * H).sum(1) + (skip * ut).abs()
            Ey = (Cx.abs() * Eh).sum(1) + (N + 3) * Yh
            if z is not None:
                f, df = silu(z[b, t])
                ef, edf = (12 + 2 * z[b, t].abs()) * f.abs(), (12 + 2 * z[b, t].abs()) * 1.1
            else:
                f, df, ef, edf = torch.ones(Dn, dtype=torch.float64), zero(Dn), zero(Dn), zero(Dn)
            v["y"][b, t], m["y"][b, t] = yh * f, Yh * f.abs()
            e["y"][b, t] = Ey * f.abs() + Yh * (ef + f.abs())
            tape.append((raw, dt, edt, a, ea, Bx, Cx, hp, Hp, Ep, h, H, Eh, yh, Yh, Ey, f, df, ef, edf))
        v["h_T"][b], m["h_T"][b], e["h_T"][b] = h, H, Eh
        if dy is None:
            continue
        g = zero(Dn, N) if dh_T is None else dh_T[b].clone()
        Gm, Eg = g.abs(), zero(Dn, N)
        for t in range(n - 1, -1, -1):
            raw, dt, edt, a, ea, Bx, Cx, hp, Hp, Ep, h, H, Eh, yh, Yh, Ey, f, df, ef, edf = tape[t]
            ut, dyt = u[b, t], dy[b, t]
            d = dyt * f
            dm, ed = d.abs(), dyt.abs() * (ef + f.abs())
            inc = Cx.abs() * dm[:, None]
            g, Gm = g + Cx * d[:, None], Gm + inc
            Eg = Eg + Cx.abs() * ed[:, None] + inc + Gm
            v["dC"][b, t], m["dC"][b, t] = fold(d[:, None] * h), fold(dm[:, None] * H)
            e["dC"][b, t] = fold(ed[:, None] * H + dm[:, None] * Eh) + (K + 1) * m["dC"][b, t]
            dtu = (dt * ut).abs()
            v["dB"][b, t] = fold(g * (dt * ut)[:, None])
            m["dB"][b, t] = fold(Gm * dtu[:, None])
            e["dB"][b, t] = fold(Eg * dtu[:, None] + Gm * (dtu * (edt + 1))[:, None]) + (K + 1) * m["dB"][b, t]
            gB, gBm = (g * Bx).sum(1), (Gm * Bx.abs()).sum(1)
            egB = (Eg * Bx.abs()).sum(1) + (N + 1) * gBm
            w, wm = g * a * hp, Gm * a * Hp
            ew = a * (Eg * Hp + Gm * Ep) + (ea + 2) * wm
            v["du"][b, t] = dt * gB + skip * d
            m["du"][b, t] = dt.abs() * gBm + (skip * d).abs()
            e["du"][b, t] = dt.abs() * (egB + edt * gBm) + skip.abs() * ed + 3 * m["du"][b, t]
            s = torch.special.expit(raw) if softplus else torch.ones_like(raw)
            es = 10 + 3 * raw.abs() if softplus else zero(Dn)
            q, qm = ut * gB + (A * w).sum(1), ut.abs() * gBm + (A.abs() * wm).sum(1)
            eq = ut.abs() * egB + (A.abs() * ew).sum(1) + (N + 5) * qm
            v["ddelta"][b, t], m["ddelta"][b, t] = q * s, qm * s
            e["ddelta"][b, t] = (eq + qm * (es + 1)) * s
            v["dA"] += dt[:, None] * w
            m["dA"] += dt[:, None].abs() * wm
            e["dA"] += dt[:, None].abs() * (ew + wm * (edt[:, None] + 1))
            v["dD"] += d * ut
            m["dD"] += dm * ut.abs()
            e["dD"] += ed * ut.abs()
            v["dz"][b, t], m["dz"][b, t] = dyt * yh * df, dyt.abs() * Yh * 1.1
            e["dz"][b, t] = dyt.abs() * (Ey * df.abs() + Yh * edf) + 3 * m["dz"][b, t]
            Eg = a * Eg + (ea + 1) * a * Gm
            g, Gm = a * g, a * Gm
        v["dh0"][b], m["dh0"][b], e["dh0"][b] = g, Gm, Eg
    v["ddelta_bias"], m["ddelta_bias"] = v["ddelta"].sum((0, 1)), m["ddelta"].sum((0, 1))
    e["ddelta_bias"] = e["ddelta"].sum((0, 1))
    for k in ("dA", "dD", "ddelta_bias"):  # sums over every token
        e[k] += (Bn * T + 2) * m[k]
    return v, m, e


def _pairs(d, rot, layout):
    i = torch.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def norm(x, w=None, kind="l2", eps=1e-6, scale=1.0, positions=None, inv_freq=None, layout="half", rscale=1.0,
         dout=None):
    """One of q, k: [B, T, H, d]. Values and magnitudes of y and, with dout, dx and dw."""
    x, w, dout = map(f64, (x, w, dout))
    B, T, H, d = x.shape
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    if rot:
        pos = torch.arange(T)[None].expand(B, T) if positions is None else positions.cpu()
        ang = pos.double()[..., None, None] * f64(inv_freq)
        c, s = torch.cos(ang), torch.sin(ang)
        p1, p2 = _pairs(d, rot, layout)

    def turn(y, back, mag=False):
        if not rot:
            return y
        out = y.clone()
        a, b_ = y[..., p1], y[..., p2]
        if mag:
            out[..., p1] = out[..., p2] = (a + b_) * abs(rscale)
        else:
            sn = -s if back else s
            out[..., p1], out[..., p2] = (a * c - b_ * sn) * rscale, (b_ * c + a * sn) * rscale
        return out

    r = torch.sqrt((x * x).sum(-1, keepdim=True)) if kind == "l2" else torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    inside = torch.zeros_like(r, dtype=torch.bool)
    if kind == "l2":
        inside = r <= eps
        r = r.clamp(min=eps)
    xh = x / r
    wn = 1.0 if w is None else w
    v, m = {}, {}
    v["y"] = turn(xh * wn, False) * scale
    m["y"] = turn((xh * wn).abs(), False, True) * abs(scale)
    if dout is not None:
        g = turn(dout, True) * scale
        gm = turn(dout.abs(), True, True) * abs(scale)
        v["dw"], m["dw"] = (g * xh).sum((0, 1, 2)), (gm * xh.abs()).sum((0, 1, 2))
        gw, gwm = g * wn, gm * abs(wn)
        n = d if kind == "rms" else 1
        dot = torch.where(inside, 0.0, (gw * xh).sum(-1, keepdim=True) / n)
        dotm = torch.where(inside, 0.0, (gwm * xh.abs()).sum(-1, keepdim=True) / n)
        v["dx"], m["dx"] = (gw - xh * dot) / r, (gwm + xh.abs() * dotm) / r
    return v, m
