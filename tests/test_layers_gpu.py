"""GPU parity of the layer operators with their 64-bit forms.

Tolerances (layers_ref.check): half a step of the result's type, and K roundings
of fp32 (2^-24) times the sum of the absolute values that enter the result. K:
  conv y     W + 1 of the taps (times |silu'| <= 1.1), 11 of the activation: 20
  conv dx    24 of silu' (its relative share of 1.1 + |p| / 2), W + 1 of the
             taps inside and outside, 1 of dX_T: 40; dweight, dbias: and one per token
  norm y     7 of the sum of squares (halved by the root), 6 of root, weight and
             scale, 15 of the rotation (angle pi, cosine 4, products): 40
  norm dx    those twice (g and xh), and 20 of the dot product: 100; dweight: and one per row
  scan       carried through the recurrence by layers_ref.scan.
"""
import pytest
import torch

import gated_delta_rule_147_b200 as gdr
import layers_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


class Rnd:
    def __init__(self, dev, seed):
        self.dev, self.g = dev, torch.Generator().manual_seed(seed)

    def __call__(self, *s, dtype=F32, scale=1.0):
        return (torch.randn(s, generator=self.g) * scale).to(dtype).to(self.dev)

    def ints(self, lo, hi, *s, dtype=torch.int64):
        return torch.randint(lo, hi, s, generator=self.g).to(dtype).to(self.dev)


def ragged(B, T, dev):
    """Lengths with an empty sequence, one token, one beyond T and a negative one."""
    vals = [T, 0, 1, T + 7, -3, max(T - 1, 0), T // 2]
    return torch.tensor([vals[i % len(vals)] for i in range(B)], dtype=torch.int32, device=dev)


def poison(x, lengths):
    """NaN in the rows behind each sequence."""
    x = x.clone()
    for b, n in enumerate(R.lens(lengths, *x.shape[:2])):
        x[b, n:] = NAN
    return x


def sliced(x, pad=8):
    """x as a slice of a wider array whose other elements are NaN."""
    wide = torch.full(x.shape[:-1] + (x.shape[-1] + 2 * pad,), NAN, dtype=x.dtype, device=x.device)
    wide[..., pad:pad + x.shape[-1]] = x
    return wide[..., pad:pad + x.shape[-1]]


# ---------------------------------------------------------------- convolution

CONV = [  # dtype, weight type, B, T, D, W, bias, state, lengths, silu, slice
    (BF, BF, 2, 70, 64, 4, True, True, False, True, 8),
    (BF, F32, 7, 37, 24, 4, False, True, True, True, 8),
    (BF, BF, 7, 9, 40, 3, True, True, True, False, 3),
    (BF, F32, 3, 1, 13, 2, True, True, False, True, 1),
    (F32, F32, 7, 33, 20, 4, True, True, True, True, 4),
    (F32, F32, 2, 131, 7, 3, False, False, False, False, 1),
    (F32, F32, 7, 2, 12, 2, True, False, True, True, 3),
    (BF, BF, 1, 3, 1, 4, True, True, False, True, 1),
    (BF, BF, 1, 0, 16, 4, True, True, False, True, 8),
    (BF, BF, 1, 4099, 8, 4, True, True, False, True, 8),
    (BF, BF, 3, 41, 22, 4, True, True, True, True, 4),
    (F32, F32, 2, 23, 18, 3, True, True, False, True, 2),
]


@pytest.mark.parametrize("dtype,wdt,B,T,D,W,bias,state,ragg,act,pad", CONV)
def test_conv(cuda_device, dtype, wdt, B, T, D, W, bias, state, ragg, act, pad):
    r = Rnd(cuda_device, B * 1000 + T + W)
    x, w = r(B, T, D, dtype=dtype), r(D, W, dtype=wdt, scale=0.6)
    b = r(D, dtype=wdt) if bias else None
    X0 = r(B, W - 1, D, dtype=dtype) if state else None
    n = ragged(B, T, cuda_device) if ragg else None
    dX = r(B, W - 1, D)
    a = "silu" if act else None
    xs = sliced(poison(x, n), pad)
    for gdt in {dtype, F32}:
        dy = r(B, T, D, dtype=gdt)
        v, m = R.conv(x, w, b, X0, n, act, dy, dX)
        y, X_T = gdr.conv_fwd(xs, w, b, X0, activation=a, lengths=n)
        R.check(y, v["y"], m["y"], 20, "y")
        assert torch.equal(X_T.double().cpu(), v["X_T"])
        g = gdr.conv_bwd(xs, w, b, X0, dy=sliced(poison(dy, n), pad), dX_T=dX, activation=a, lengths=n)
        R.check(g["dx"], v["dx"], m["dx"], 40, "dx")
        R.check(g["dweight"], v["dweight"], m["dweight"], 40 + B * T, "dweight")
        assert (g["dbias"] is None) == (b is None) and (g["dX0"] is None) == (X0 is None)
        if bias:
            R.check(g["dbias"], v["dbias"], m["dbias"], 40 + B * T, "dbias")
        if state:
            R.check(g["dX0"], v["dX0"], m["dX0"], 40, "dX0")
    g2 = gdr.conv_bwd(xs, w, b, X0, dy=dy, activation=a, lengths=n, need_dX0=False)
    v, m = R.conv(x, w, b, X0, n, act, dy)
    assert g2["dX0"] is None
    R.check(g2["dx"], v["dx"], m["dx"], 40, "dx without dX_T")


@pytest.mark.parametrize("dtype,D,W", [(BF, 64, 4), (BF, 5, 3), (F32, 8, 2), (F32, 9, 4), (BF, 30, 4)])
def test_conv_steps_continue_the_sequence(cuda_device, dtype, D, W):
    """Prompt, then single tokens from the carried rows: bit for bit the whole
    sequence's outputs; the state may be carried in place."""
    r = Rnd(cuda_device, D)
    x, w, b = r(3, 20, D, dtype=dtype), r(D, W, dtype=dtype), r(D, dtype=dtype)
    X = r(3, W - 1, D, dtype=dtype)
    whole, X_T = gdr.conv_fwd(x, w, b, X)
    y, X1 = gdr.conv_fwd(x[:, :1], w, b, X, X_T=X)
    assert X1 is X and torch.equal(y, whole[:, :1])
    for t in range(1, 20):
        assert torch.equal(gdr.conv_step(x[:, t], w, b, X), whole[:, t])
    assert torch.equal(X, X_T)
    assert gdr.conv_fwd(x, w, b, X, final_state=False)[1] is None


@pytest.mark.parametrize("dtype,B,D", [(BF, 203, 12288), (F32, 810, 2999)])
def test_conv_step_of_a_large_batch(cuda_device, dtype, B, D):
    """Several sequences to a thread, the last thread with fewer: the same as a
    prompt of one token."""
    r = Rnd(cuda_device, B)
    x, w, b, X = r(B, D, dtype=dtype), r(D, 4, dtype=dtype), r(D, dtype=dtype), r(B, 3, D, dtype=dtype)
    y, X_T = gdr.conv_fwd(x[:, None], w, b, X)
    assert torch.equal(gdr.conv_step(x, w, b, X), y[:, 0]) and torch.equal(X, X_T)


def test_conv_extremes(cuda_device):
    """Inputs whose activation saturates: no NaN, the limits of silu."""
    x = torch.tensor([1e30, -1e30, 200.0, -200.0, 0.0], device=cuda_device)[None, :, None].repeat(1, 1, 4)
    w = torch.tensor([[0.0, 1.0]], device=cuda_device).repeat(4, 1)
    y, _ = gdr.conv_fwd(x, w)
    assert torch.allclose(y[0, :, 0].cpu(), torch.tensor([1e30, 0.0, 200.0, 0.0, 0.0]), rtol=1e-6, atol=1e-37)
    g = gdr.conv_bwd(x[:, 2:], w, dy=torch.ones_like(x[:, 2:]))
    assert torch.allclose(g["dx"][0, :, 0].cpu(), torch.tensor([1.0, 0.0, 0.5]), atol=1e-6)


# ---------------------------------------------------------------- selective scan

SCAN = [  # dtype, B, T, D, N, G, softplus, gate, skip, bias, state, lengths, slice
    (BF, 2, 70, 64, 16, 1, True, True, True, True, True, False, 8),
    (F32, 2, 61, 40, 16, 2, True, True, True, True, True, False, 5),
    (BF, 7, 19, 33, 16, 3, True, True, True, True, True, True, 3),
    (F32, 7, 33, 12, 5, 1, False, False, False, False, False, True, 1),
    (BF, 1, 130, 24, 64, 2, True, True, False, True, True, False, 8),
    (F32, 2, 17, 6, 128, 1, True, False, True, False, True, False, 2),
    (F32, 3, 1, 17, 4, 1, True, True, True, True, True, False, 1),
    (F32, 3, 40, 70, 1, 1, True, True, True, True, True, True, 1),
    (BF, 2, 40, 16, 24, 4, False, True, True, True, False, False, 8),
    (F32, 2, 0, 8, 8, 1, True, True, True, True, True, False, 4),
    (F32, 1, 700, 3, 8, 1, True, False, True, True, True, False, 1),
    (BF, 1, 1043, 40, 16, 1, True, True, True, True, True, False, 8),
    (F32, 3, 800, 9, 6, 1, True, True, True, True, True, True, 1),
    (BF, 2, 50, 300, 4, 1, True, True, True, True, True, False, 8),
    (BF, 3, 43, 76, 6, 2, True, True, True, True, True, True, 2),
    (BF, 1, 600, 22, 16, 1, True, True, True, True, True, False, 2),
    (F32, 2, 45, 35, 10, 1, True, True, True, True, True, False, 1),
]


def scan_inputs(r, dtype, B, T, D, N, G, softplus, gate, skip, bias, state):
    A = -torch.exp(r(D, N))
    delta = r(B, T, D, dtype=dtype, scale=0.5) if softplus else r(B, T, D, scale=0.3).abs().to(dtype)
    return dict(u=r(B, T, D, dtype=dtype), delta=delta, A=A, Bm=r(B, T, G, N, dtype=dtype),
                Cm=r(B, T, G, N, dtype=dtype), D=r(D) if skip else None,
                z=r(B, T, D, dtype=dtype, scale=2.0) if gate else None, h0=r(B, D, N) if state else None,
                delta_bias=(r(D) - 1 if softplus else r(D).abs() * 0.1) if bias else None)


def check_scan(got, ref, names):
    v, m, e = ref
    for k in names:
        R.check(got[k], v[k], e[k], 1, k)


@pytest.mark.parametrize("dtype,B,T,D,N,G,softplus,gate,skip,bias,state,ragg,pad", SCAN)
def test_scan(cuda_device, dtype, B, T, D, N, G, softplus, gate, skip, bias, state, ragg, pad):
    r = Rnd(cuda_device, B * 1000 + T + N)
    i = scan_inputs(r, dtype, B, T, D, N, G, softplus, gate, skip, bias, state)
    n = ragged(B, T, cuda_device) if ragg else None
    dh = r(B, D, N)
    kw = dict(delta_bias=i["delta_bias"], delta_softplus=softplus, lengths=n)
    masked = lambda t: None if t is None else sliced(poison(t, n), pad)  # noqa: E731
    BC = sliced(poison(torch.cat([i["Bm"].flatten(2), i["Cm"].flatten(2)], -1), n), pad)
    Bm, Cm = (BC[..., k * G * N:(k + 1) * G * N].unflatten(-1, (G, N)) for k in (0, 1))
    args = (masked(i["u"]), masked(i["delta"]), i["A"], Bm, Cm, i["D"], masked(i["z"]), i["h0"])
    for gdt in {dtype, F32}:
        dy = r(B, T, D, dtype=gdt)
        ref = R.scan(i["u"], i["delta"], i["A"], i["Bm"], i["Cm"], i["D"], i["z"], i["h0"], i["delta_bias"], softplus,
                     n, dy, dh)
        y, h_T = gdr.scan_fwd(*args, **kw)
        check_scan({"y": y, "h_T": h_T}, ref, ("y", "h_T"))
        g = gdr.scan_bwd(*args, dy=masked(dy), dh_T=dh, **kw)
        for k, src in (("dD", "D"), ("dz", "z"), ("ddelta_bias", "delta_bias"), ("dh0", "h0")):
            assert (g[k] is None) == (i[src] is None)
        check_scan(g, ref, [k for k in g if g[k] is not None])
    ref = R.scan(i["u"], i["delta"], i["A"], i["Bm"], i["Cm"], i["D"], i["z"], i["h0"], i["delta_bias"], softplus, n,
                 dy)
    g = gdr.scan_bwd(*args, dy=dy, need_dh0=False, **kw)
    assert g["dh0"] is None
    check_scan(g, ref, ("du", "ddelta", "dA", "dB", "dC"))


def test_scan_split_workspace(cuda_device):
    """The split of the tokens needs a workspace; without one, or with one too
    small, the call runs unsplit, with the same results up to rounding."""
    r = Rnd(cuda_device, 77)
    B, T, D, N = 1, 1500, 24, 16
    i = scan_inputs(r, F32, B, T, D, N, 1, True, True, True, True, True)
    args = tuple(i[k] for k in ("u", "delta", "A", "Bm", "Cm", "D", "z", "h0"))
    kw = dict(delta_bias=i["delta_bias"], delta_softplus=True)
    ref = R.scan(*args, i["delta_bias"], True)
    got = {}
    for name, ws in (("auto", "auto"), ("none", None), ("small", torch.empty(256, dtype=torch.uint8, device=cuda_device))):
        got[name] = gdr.scan_fwd(*args, workspace=ws, **kw)
        check_scan(dict(zip(("y", "h_T"), got[name])), ref, ("y", "h_T"))
    assert torch.equal(got["none"][0], got["small"][0]) and torch.equal(got["none"][1], got["small"][1])
    for n in (None, torch.tensor([700], dtype=torch.int32, device=cuda_device)):  # the state carried in place
        want = gdr.scan_fwd(*args, lengths=n, **kw)
        h = i["h0"].clone()
        y, h_T = gdr.scan_fwd(*args[:-1], h, h_T=h, lengths=n, **kw)
        assert h_T is h and torch.equal(h, want[1]) and torch.equal(y, want[0])


@pytest.mark.parametrize("dtype,D,N,G", [(BF, 48, 16, 1), (F32, 10, 7, 2), (BF, 4, 128, 1), (F32, 33, 4, 1)])
def test_scan_steps_continue_the_sequence(cuda_device, dtype, D, N, G):
    """A prompt's final state carried on by single tokens."""
    r = Rnd(cuda_device, D)
    B, T, P = 2, 24, 17
    i = scan_inputs(r, dtype, B, T, D, N, G, True, True, True, True, True)
    ref = R.scan(*(i[k] for k in ("u", "delta", "A", "Bm", "Cm", "D", "z", "h0", "delta_bias")), True)
    kw = dict(delta_bias=i["delta_bias"], delta_softplus=True)
    seq = ("u", "delta", "Bm", "Cm", "z")
    cut = {k: (v[:, :P] if k in seq else v) for k, v in i.items()}
    h = i["h0"].clone()
    _, h1 = gdr.scan_fwd(*(cut[k] for k in ("u", "delta", "A", "Bm", "Cm", "D", "z")), h, h_T=h, **kw)
    assert h1 is h
    for t in range(P, T):
        s = {k: (v[:, t] if k in seq else v) for k, v in i.items()}
        y = gdr.scan_step(*(s[k] for k in ("u", "delta", "A", "Bm", "Cm", "D", "z")), h, **kw)
        R.check(y, ref[0]["y"][:, t], ref[2]["y"][:, t], 1, f"token {t}")
    R.check(h, ref[0]["h_T"], ref[2]["h_T"], 1, "h")


def test_scan_extremes(cuda_device):
    """Decays of 0 (A = -inf and steps that underflow), steps near 0 and none
    (large negative delta), and no state lost over them."""
    B, T, D, N = 1, 21, 8, 4
    r = Rnd(cuda_device, 5)
    u, Bm, Cm = r(B, T, D), r(B, T, 1, N), r(B, T, 1, N)
    A = torch.tensor([-float("inf"), -1e30, -1.0, 0.0], device=cuda_device).repeat(D, 1)
    delta = torch.full((B, T, D), -200.0, device=cuda_device)  # softplus = 0: every token keeps the state
    h0 = r(B, D, N)
    y, h = gdr.scan_fwd(u, delta, A, Bm, Cm, None, None, h0, delta_softplus=True)
    assert torch.equal(h, h0)
    want = (Cm[0, :, 0, None, :].double() * h0[0].double()).sum(-1)
    assert torch.allclose(y[0].double(), want, rtol=0, atol=8 * 2.0 ** -24 * 20)
    h = h0.clone()
    gdr.scan_step(u[:, 0], delta[:, 0], A, Bm[:, 0], Cm[:, 0], None, None, h, delta_softplus=True)
    assert torch.equal(h, h0)
    n = torch.tensor([13], dtype=torch.int32, device=cuda_device)
    y, h = gdr.scan_fwd(u, torch.ones_like(delta), A, Bm, Cm, None, None, h0, lengths=n)
    last = u[0, 12, :, None] * Bm[0, 12, 0]
    assert torch.equal(h[0, :, :2], last[:, :2]) and not torch.isnan(y).any() and (y[0, 13:] == 0).all()
    g = gdr.scan_bwd(u, torch.ones_like(delta), A, Bm, Cm, None, None, h0, dy=torch.ones_like(u), lengths=n)
    assert (g["dh0"][..., :2] == 0).all() and not any(torch.isnan(t).any() for k, t in g.items() if t is not None and
                                                      k not in ("ddelta", "dA"))


# ---------------------------------------------------------------- norm and rotation

NORM = [  # dtype, weight type, grad type, B, T, Hq, Hk, d, rot, layout, kind, positions, scale
    (BF, None, BF, 2, 33, 4, 2, 128, 128, "half", "l2", None, 0.09),
    (BF, BF, F32, 2, 17, 3, 3, 256, 64, "interleaved", "rms", torch.int64, 1.0),
    (F32, F32, F32, 3, 5, 8, 2, 64, 32, "half", "rms", torch.int32, 0.125),
    (BF, F32, BF, 1, 40, 5, 1, 72, 36, "half", "rms", torch.int64, 1.0),
    (F32, None, F32, 2, 9, 2, 1, 19, 18, "interleaved", "l2", torch.int64, 1.0),
    (F32, F32, F32, 1, 1, 1, 1, 1, 0, "half", "rms", None, 1.0),
    (BF, None, BF, 300, 1, 16, 4, 128, 64, "half", "l2", torch.int32, 1.0),
    (BF, BF, BF, 1, 700, 2, 2, 16, 16, "half", "rms", None, 1.0),
    (BF, None, F32, 1, 7, 3, 0, 200, 0, "half", "l2", None, 2.0),
    (F32, None, F32, 1, 3, 40, 40, 255, 254, "half", "rms", None, 1.0),
    (BF, BF, BF, 2, 21, 3, 2, 104, 104, "half", "rms", torch.int64, 1.0),
    (BF, None, F32, 3, 9, 5, 1, 24, 12, "half", "l2", torch.int32, 1.0),
    (F32, F32, F32, 2, 13, 2, 2, 256, 250, "half", "rms", None, 0.5),
    (BF, BF, BF, 2, 11, 2, 1, 114, 56, "half", "rms", torch.int64, 1.0),
    (BF, None, BF, 1, 50, 3, 3, 30, 30, "interleaved", "l2", None, 1.0),
]


@pytest.mark.parametrize("dtype,wdt,gdt,B,T,Hq,Hk,d,rot,layout,kind,pos,qs", NORM)
def test_norm(cuda_device, dtype, wdt, gdt, B, T, Hq, Hk, d, rot, layout, kind, pos, qs):
    r = Rnd(cuda_device, B * 1000 + T + d)
    qkv = r(B, T, (Hq + 2 * Hk) * d, dtype=dtype, scale=3.0)
    q, k = qkv[..., :Hq * d].unflatten(-1, (Hq, d)), qkv[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d)) if Hk else None
    qw, kw = (r(d, dtype=wdt), r(d, dtype=wdt) if Hk else None) if wdt else (None, None)
    f = torch.exp(-torch.arange(rot // 2) / 3.0).to(cuda_device) if rot else None
    p = None if pos is None or not rot else r.ints(-(1 << 22), 1 << 22, B, T, dtype=pos)
    dq, dk = r(B, T, Hq, d, dtype=gdt), r(B, T, Hk, d, dtype=gdt) if Hk else None
    kws = dict(kind=kind, eps=1e-5, q_scale=qs, positions=p, inv_freq=f, rotary=layout, rotary_scale=1.25)
    yq, yk = gdr.qk_norm_fwd(q, k, qw, kw, **kws)
    g = gdr.qk_norm_bwd(q, k, qw, kw, dq=dq, dk=dk, **kws)
    assert (yk is None) == (Hk == 0) and (g["dk"] is None) == (Hk == 0)
    for x, w, y, do, n, s, H in ((q, qw, yq, dq, "q", qs, Hq), (k, kw, yk, dk, "k", 1.0, Hk)):
        if x is None:
            continue
        v, m = R.norm(x, w, kind, 1e-5, s, p, f, layout, 1.25, do)
        R.check(y, v["y"], m["y"], 40, n)
        R.check(g["d" + n], v["dx"], m["dx"], 100, "d" + n)
        assert (g[f"d{n}_weight"] is None) == (w is None)
        if w is not None:
            R.check(g[f"d{n}_weight"], v["dw"], m["dw"], 100 + B * T * H, f"d{n}_weight")
    if Hk:  # in place over dense inputs
        qc, kc = q.contiguous(), k.contiguous()
        gdr.qk_norm_fwd(qc, kc, qw, kw, q_out=qc, k_out=kc, **kws)
        assert torch.equal(qc, yq) and torch.equal(kc, yk)


@pytest.mark.parametrize("d,pad", [(72, 0), (66, 0), (67, 1), (120, 0)])
@pytest.mark.parametrize("layout,rot", [("half", 0), ("half", 32), ("interleaved", 32)])
def test_norm_of_rows_narrower_than_their_lanes(cuda_device, d, pad, layout, rot):
    """What an earlier call left in shared memory (here NaN weights of wider rows
    on as many lanes) does not reach a row."""
    r = Rnd(cuda_device, d)
    f = torch.exp(-torch.arange(rot // 2) / 3.0).to(cuda_device) if rot else None
    kws = dict(kind="rms", eps=1e-5, inv_freq=f, rotary=layout)
    wide, bad = r(1, 2048, 1, 128 + pad)[..., :128], torch.full((128,), NAN, device=cuda_device)
    if d % 8:  # rows that are no whole vectors either
        wide = sliced(wide, 1)
    q, k, dq, dk = (r(2, 300, 2, d + pad)[..., :d] for _ in range(4))
    qw, kw = r(d), r(d)
    gdr.qk_norm_bwd(wide, q_weight=bad, dq=wide, **kws)
    g = gdr.qk_norm_bwd(q, k, qw, kw, dq=dq, dk=dk, **kws)
    gdr.qk_norm_fwd(wide, q_weight=bad, **kws)
    yq, yk = gdr.qk_norm_fwd(q, k, qw, kw, **kws)
    for x, w, y, do, n in ((q, qw, yq, dq, "q"), (k, kw, yk, dk, "k")):
        v, m = R.norm(x, w, "rms", 1e-5, 1.0, None, f, layout, 1.0, do)
        R.check(y, v["y"], m["y"], 40, n)
        R.check(g["d" + n], v["dx"], m["dx"], 100, "d" + n)
        R.check(g[f"d{n}_weight"], v["dw"], m["dw"], 100 + 2 * 300 * 2, f"d{n}_weight")


@pytest.mark.parametrize("kind", ["l2", "rms"])
def test_norm_zero_and_tiny_rows(cuda_device, kind):
    """Rows of zeros and rows below eps: finite values and gradients."""
    x = torch.zeros(1, 3, 1, 16, device=cuda_device)
    x[0, 1] = 1e-9
    x[0, 2] = 1e-30
    dy = torch.ones_like(x)
    y, _ = gdr.qk_norm_fwd(x, kind=kind, eps=1e-6)
    g = gdr.qk_norm_bwd(x, dq=dy, kind=kind, eps=1e-6)["dq"]
    v, m = R.norm(x, None, kind, 1e-6, dout=dy)
    R.check(y, v["y"], m["y"], 40, "y")
    R.check(g, v["dx"], m["dx"], 100, "dx")


def test_norm_far_positions(cuda_device):
    """At position 2^33 the angle's error is that of f / (2 pi) as a 53-bit number:
    2^-53 of 2^33 / 2 radians, 2^-21, 8 units beside the usual 40."""
    d = 16
    q = Rnd(cuda_device, 3)(1, 1, 1, d)
    f = torch.full((d // 2,), 0.5, device=cuda_device)
    far = torch.tensor([[1 << 33]], device=cuda_device)
    y, _ = gdr.qk_norm_fwd(q, positions=far, inv_freq=f)
    v, m = R.norm(q, inv_freq=f, positions=far)
    R.check(y, v["y"], m["y"], 48, "y")


# ---------------------------------------------------------------- together

def test_layer_forward_backward_and_decode(cuda_device):
    """Convolution, norm and the delta rule as one layer: forward, its gradients
    against a 64-bit autograd of the same formulas, and decode that continues it."""
    r = Rnd(cuda_device, 11)
    B, T, H, d, W = 2, 65, 2, 32, 4
    D = 3 * H * d
    x, w, X0 = r(B, T + 4, D), r(D, W, scale=0.5), torch.zeros(B, W - 1, D, device=cuda_device)
    alpha = torch.sigmoid(r(B, T + 4, H) + 3)
    beta = torch.sigmoid(r(B, T + 4, H))
    f = (100.0 ** (-torch.arange(d // 2) / (d // 2))).to(cuda_device)
    kw = dict(kind="l2", q_scale=d ** -0.5, inv_freq=f)
    dO = r(B, T, H, d)

    def heads(y, i):
        return y[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d))

    def formulas(x, w, a, b):
        rows = torch.cat([torch.zeros(B, W - 1, D, dtype=torch.float64), x], 1)
        y = torch.nn.functional.silu(sum(w[:, j] * rows[:, j:j + x.shape[1]] for j in range(W)))
        ang = torch.arange(x.shape[1], dtype=torch.float64)[:, None, None] * f.double().cpu()
        unit = torch.polar(torch.ones_like(ang), ang)

        def turn(v):
            v = v / v.norm(dim=-1, keepdim=True)
            c = torch.complex(v[..., :d // 2], v[..., d // 2:]) * unit
            return torch.cat([c.real, c.imag], -1)
        q, k, v = turn(heads(y, 0)) * d ** -0.5, turn(heads(y, 1)), heads(y, 2)
        S, o = torch.zeros(B, H, d, d, dtype=torch.float64), []
        for t in range(x.shape[1]):
            kt, bt = k[:, t], b[:, t, :, None]
            S = a[:, t, :, None, None] * S
            S = S + (bt * kt)[..., None] * (v[:, t] - (kt[..., None] * S).sum(-2))[..., None, :]
            o.append((q[:, t, ..., None] * S).sum(-2))
        return torch.stack(o, 1)

    leaves = [t.double().cpu().requires_grad_() for t in (x[:, :T], w, alpha[:, :T], beta[:, :T])]
    o_ref = formulas(*leaves)
    want = torch.autograd.grad((o_ref * R.f64(dO)).sum(), leaves)

    y, X = gdr.conv_fwd(x[:, :T], w, None, X0)
    q, k = gdr.qk_norm_fwd(heads(y, 0), heads(y, 1), **kw)
    v = heads(y, 2).contiguous()
    a, b = alpha[:, :T].contiguous(), beta[:, :T].contiguous()
    o, S = gdr.chunk_fwd(q, k, v, a, b, gdr.TIED)
    g = gdr.chunk_bwd(q, k, v, a, b, gdr.TIED, dO=dO, need_dS0=False)
    gn = gdr.qk_norm_bwd(heads(y, 0), heads(y, 1), dq=g["dq"], dk=g["dk"], **kw)
    dy = torch.cat([gn["dq"].flatten(2), gn["dk"].flatten(2), g["dv"].flatten(2)], -1)
    gc = gdr.conv_bwd(x[:, :T], w, None, X0, dy=dy)
    for got, ref, what in ((o, o_ref.detach(), "o"), (gc["dx"], want[0], "dx"), (gc["dweight"], want[1], "dweight"),
                           (g["dalpha"], want[2], "dalpha"), (g["db"], want[3], "dbeta")):
        err = (got.double().cpu() - ref).abs().max() / ref.abs().max()
        # the recurrence's fp32 bound; the operators around it add tens of 2^-24
        assert err <= 1e-4, (what, err)

    whole = formulas(R.f64(x), R.f64(w), R.f64(alpha), R.f64(beta))
    for t in range(T, T + 4):
        yt = gdr.conv_step(x[:, t], w, None, X)
        pos = torch.full((B, 1), t, device=cuda_device)
        qt, kt = gdr.qk_norm_fwd(heads(yt[:, None], 0), heads(yt[:, None], 1), positions=pos, **kw)
        ot = gdr.decode_step(qt[:, 0], kt[:, 0], heads(yt, 2).contiguous(), alpha[:, t].contiguous(),
                             beta[:, t].contiguous(), gdr.TIED, S)
        assert (ot.double().cpu() - whole[:, t]).abs().max() / whole.abs().max() <= 1e-4, t


def test_conv_into_scan(cuda_device):
    """The scan's layer: u through the convolution, forward and backward, ragged."""
    r = Rnd(cuda_device, 12)
    B, T, D, N, W = 3, 29, 24, 8, 4
    x, w, b, X0 = r(B, T, D), r(D, W, scale=0.5), r(D), r(B, W - 1, D)
    n = torch.tensor([29, 1, 14], dtype=torch.int32, device=cuda_device)
    i = scan_inputs(r, F32, B, T, D, N, 1, True, True, True, True, True)
    kw = dict(delta_bias=i["delta_bias"], delta_softplus=True, lengths=n)
    rest = tuple(i[k] for k in ("delta", "A", "Bm", "Cm", "D", "z", "h0"))
    dy = r(B, T, D)
    u, _ = gdr.conv_fwd(x, w, b, X0, lengths=n)
    y, _ = gdr.scan_fwd(u, *rest, **kw)
    g = gdr.scan_bwd(u, *rest, dy=dy, **kw)
    gc = gdr.conv_bwd(x, w, b, X0, dy=g["du"], lengths=n)
    u64 = R.conv(x, w, b, X0, n)[0]["y"]
    v, _, _ = R.scan(u64, *rest, i["delta_bias"], True, n, dy)
    c, _ = R.conv(x, w, b, X0, n, True, v["du"])
    for got, ref in ((y, v["y"]), (gc["dx"], c["dx"]), (gc["dweight"], c["dweight"]), (gc["dX0"], c["dX0"])):
        assert (got.double().cpu() - ref).abs().max() <= 1e-5 * ref.abs().max()


def _calls(r, big):
    """One closure per operator, over tensors of its own."""
    B, T, D, N, W = (4, 515, 136, 16, 4) if big else (1, 5, 8, 4, 3)
    i = scan_inputs(r, BF, B, T, D, N, 1, True, True, True, True, True)
    sa = tuple(i[k] for k in ("u", "delta", "A", "Bm", "Cm", "D", "z", "h0"))
    kw = dict(delta_bias=i["delta_bias"], delta_softplus=True)
    x, w, b, X0 = r(B, T, D, dtype=BF), r(D, W, dtype=BF), r(D, dtype=BF), r(B, W - 1, D, dtype=BF)
    q, k, nw = r(B, T, 4, 64, dtype=BF), r(B, T, 2, 64, dtype=BF), r(64, dtype=BF)
    f = torch.full((16,), 0.1, device=r.dev)
    dy, dq, dk = r(B, T, D), r(B, T, 4, 64), r(B, T, 2, 64)
    nk = dict(kind="rms", inv_freq=f)
    one = tuple(t[:, 0] if t.dim() > 2 and t.shape[1] == T else t for t in sa[:7])
    return [lambda **s: gdr.conv_fwd(x, w, b, X0, **s), lambda **s: gdr.conv_bwd(x, w, b, X0, dy=dy, **s),
            lambda **s: (gdr.conv_step(x[:, 0], w, b, X0.clone(), **s),),
            lambda **s: gdr.scan_fwd(*sa, **kw, **s), lambda **s: gdr.scan_bwd(*sa, dy=dy, **kw, **s),
            lambda **s: (gdr.scan_step(*one, sa[7].clone(), **kw, **s),),
            lambda **s: gdr.qk_norm_fwd(q, k, nw, nw, **nk, **s),
            lambda **s: gdr.qk_norm_bwd(q, k, nw, nw, dq=dq, dk=dk, **nk, **s)]


def _flat(o):
    return [t for t in (o.values() if isinstance(o, dict) else o) if t is not None]


@pytest.mark.parametrize("big", [True, False])
def test_repeatable_captured_and_on_another_stream(cuda_device, big):
    """Bit for bit the same: twice, from a replayed graph (two graphs at once),
    on a stream given or current."""
    calls = _calls(Rnd(cuda_device, 21), big)
    first = [_flat(c()) for c in calls]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                outs = [_flat(c()) for c in calls]
        graphs.append((g, outs))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    given = [_flat(c(stream=side)) for c in calls[:2] + calls[3:5] + calls[6:]]
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.stream(side):
        inside = [_flat(c()) for c in calls]
    torch.cuda.synchronize()
    for got in [o for _, o in graphs] + [inside, [_flat(c()) for c in calls]]:
        for a, b in zip(first, got):
            assert all(torch.equal(s, t) for s, t in zip(a, b)) and len(a) == len(b)
    for a, b in zip(first[:2] + first[3:5] + first[6:], given):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_offsets_beyond_32_bits(cuda_device):
    """Batch rows more than 2^31 elements apart: the last equals the same row alone."""
    B, T, D, N = 2, 40, 32, 16
    r = Rnd(cuda_device, 31)
    far = torch.empty((1 << 31) + (1 << 20), dtype=BF, device=cuda_device)

    def spread(t):  # t [B, ...] with its last batch row 2^31 elements on
        at = spread.at
        spread.at += t[0].numel() + 64
        v = torch.as_strided(far, t.shape, (1 << 31,) + t.stride()[1:], at)
        v.copy_(t)
        return v
    spread.at = 0
    i = scan_inputs(r, BF, B, T, D, N, 1, True, True, True, True, True)
    w, q, k = r(D, 4, dtype=BF), r(B, T, 2, 16, dtype=BF), r(B, T, 1, 16, dtype=BF)
    dy = r(B, T, D, dtype=BF)
    kw = dict(delta_bias=i["delta_bias"], delta_softplus=True)
    sa = [i[k_] for k_ in ("u", "delta", "A", "Bm", "Cm", "D", "z", "h0")]
    sb = [spread(t) if k_ in (0, 1, 3, 4, 6) else t for k_, t in enumerate(sa)]
    far_dy, far_q, far_k = spread(dy), spread(q), spread(k)
    pairs = [(gdr.conv_fwd(sa[0], w), gdr.conv_fwd(sb[0], w)),
             (gdr.conv_bwd(sa[0], w, dy=dy), gdr.conv_bwd(sb[0], w, dy=far_dy)),
             (gdr.scan_fwd(*sa, **kw), gdr.scan_fwd(*sb, **kw)),
             (gdr.scan_bwd(*sa, dy=dy, **kw), gdr.scan_bwd(*sb, dy=far_dy, **kw)),
             (gdr.qk_norm_fwd(q, k), gdr.qk_norm_fwd(far_q, far_k)),
             (gdr.qk_norm_bwd(q, k, dq=q, dk=k), gdr.qk_norm_bwd(far_q, far_k, dq=far_q, dk=far_k))]
    torch.cuda.synchronize()
    for a, b in pairs:
        assert all(torch.equal(s, t) for s, t in zip(_flat(a), _flat(b)))
