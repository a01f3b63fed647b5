"""The layer operators at the ends of their ranges: steps that mask a token,
values that are not finite, the longest sums, the most rows."""
import pytest
import torch

import gated_delta_rule_147_b200 as gdr
import layers_ref as R
from test_layers_gpu import Rnd, scan_inputs

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
SEQ = ("u", "delta", "Bm", "Cm", "z")
ARGS = ("u", "delta", "A", "Bm", "Cm", "D", "z", "h0")


def same(a, b):
    return torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) and torch.equal(a.isnan(), b.isnan())


# ---------------------------------------------------------------- selective scan

@pytest.mark.parametrize("dtype,B,T,D,N,G", [(F32, 2, 37, 12, 16, 1), (BF, 2, 70, 24, 4, 2), (BF, 1, 1030, 8, 16, 1),
                                             (F32, 1, 600, 5, 3, 1)])
@pytest.mark.parametrize("low", ["-inf", "lowest"])
def test_scan_steps_that_mask_a_token(cuda_device, dtype, B, T, D, N, G, low):
    """A step input of -inf, or the type's lowest number, is a step of 0: the token
    keeps the state and has no gradient through it. Bit for bit what an input of
    -200 gives (e^-200 is 0 in fp32), which the 64-bit form checks; the same in
    prompts (also split ones), gradients and single tokens."""
    r = Rnd(cuda_device, T + N)
    i = scan_inputs(r, dtype, B, T, D, N, G, True, True, True, True, True)
    masked = torch.zeros(B, T, D, dtype=torch.bool, device=cuda_device)
    masked[:, 3::5] = True
    masked[0, T // 2:T // 2 + 20] = True
    masked[:, 0, ::2] = True
    dy, dh = r(B, T, D), r(B, D, N)
    kw = dict(delta_bias=i["delta_bias"], delta_softplus=True)
    got = []
    for v in (-200.0, -INF if low == "-inf" else torch.finfo(dtype).min):
        a = dict(i, delta=torch.where(masked, torch.tensor(v, dtype=dtype, device=cuda_device), i["delta"]))
        args = tuple(a[k] for k in ARGS)
        y, h_T = gdr.scan_fwd(*args, **kw)
        g = gdr.scan_bwd(*args, dy=dy, dh_T=dh, **kw)
        h = i["h0"].clone()
        steps = [gdr.scan_step(*(None if a[k] is None else a[k][:, t] if k in SEQ else a[k] for k in ARGS[:7]), h, **kw)
                 for t in range(min(T, 24))]
        got.append(dict(g, y=y, h_T=h_T, h=h, steps=torch.stack(steps, 1), whole=gdr.scan_fwd(*args, workspace=None, **kw)[0]))
        if v == -200.0:
            ref = R.scan(*args, i["delta_bias"], True, None, dy, dh)
            for k in ref[0]:
                R.check(got[0][k], ref[0][k], ref[2][k], 1, k)
    for k, v in got[0].items():
        assert torch.equal(v, got[1][k]), k
    assert (got[1]["ddelta"][masked] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_scan_steps_at_the_upper_end(cuda_device, dtype):
    """Huge and infinite steps, and NaN: softplus is the identity there; a prompt of one
    token and a single token agree, and a NaN stays with its channel."""
    B, D, N = 1, 8, 4
    r = Rnd(cuda_device, 9)
    i = scan_inputs(r, dtype, B, 1, D, N, 1, True, False, True, False, True)
    i["u"] = i["u"] * 1e-30
    for v in (1e10, 3e38, INF, NAN):
        delta = i["delta"].clone()
        delta[..., ::2] = v
        args = (i["u"], delta, i["A"], i["Bm"], i["Cm"], i["D"], None)
        y, h = gdr.scan_fwd(*args, i["h0"], delta_softplus=True)
        h1 = i["h0"].clone()
        y1 = gdr.scan_step(*(t[:, 0] if k in SEQ and t is not None else t for k, t in zip(ARGS, args)), h1,
                           delta_softplus=True)
        assert torch.equal(h.isnan(), h1.isnan()) and torch.equal(y[:, 0].isnan(), y1.isnan())
        assert torch.isfinite(h[:, 1::2]).all() and torch.isfinite(y[..., 1::2]).all()
        if v != v:
            assert h[:, ::2].isnan().all()
        else:
            dtu = v * i["u"].double()[:, 0, ::2, None] if v == INF else delta.double()[:, 0, ::2, None] * i["u"].double()[:, 0, ::2, None]
            want = (dtu * i["Bm"].double()[:, 0]).float()  # the decay is 0
            for got in (h, h1):
                ok = (got[:, ::2] == want) | ((got[:, ::2] - want).abs() <= 4 * R.U32 * want.abs())
                assert ok.all()


@pytest.mark.parametrize("N", [4, 7, 16, 40])
def test_scan_nan_decay_shows_in_every_call(cuda_device, N):
    """A NaN in A reaches the state and the outputs of its channel, and no other, in a
    prompt and in a single token alike."""
    B, D = 2, 12
    r = Rnd(cuda_device, N)
    i = scan_inputs(r, F32, B, 1, D, N, 1, True, True, True, True, True)
    i["A"][5, N - 1] = NAN
    i["A"][7, 0] = NAN
    bad = torch.zeros(D, dtype=torch.bool, device=cuda_device)
    bad[[5, 7]] = True
    kw = dict(delta_bias=i["delta_bias"], delta_softplus=True)
    y, h = gdr.scan_fwd(*(i[k] for k in ARGS), **kw)
    h1 = i["h0"].clone()
    y1 = gdr.scan_step(*(i[k][:, 0] if k in SEQ else i[k] for k in ARGS[:7]), h1, **kw)
    for y_, h_ in ((y[:, 0], h), (y1, h1)):
        assert torch.equal(y_.isnan(), bad.expand(B, D)) and torch.equal(h_.isnan(), i["A"].isnan().expand(B, D, N))


def test_scan_skip_gradient_of_a_long_sum(cuda_device):
    """dD of 4096 tokens, 512 a thread. Every term is 1 + 63 2^-23, which a sum of 128
    terms and more loses at every addition (94 2^-24 in all). With compensated sums
    2 roundings remain, of 8 threads' sums 4.5, of 2 sequences 1.5."""
    B, T, D, N = 2, 4096, 9600, 16
    v = 1 + 63 * 2.0 ** -23
    u, delta, dy = (torch.full((1, 1, D), c, device=cuda_device).expand(B, T, D) for c in (1.0, 0.1, v))
    none = torch.zeros(1, 1, 1, N, device=cuda_device).expand(B, T, 1, N)
    g = gdr.scan_bwd(u, delta, -torch.ones(D, N, device=cuda_device), none, none, torch.ones(D, device=cuda_device), dy=dy)
    off = ((g["dD"].double() - B * T * v).abs().max() / (B * T * v)).item()
    assert off <= 8 * R.U32, off / R.U32


def test_scan_skip_gradient_that_overflows(cuda_device):
    """An infinite sum stays infinite, and with its channel."""
    T, D, N = 40, 8, 4
    r = Rnd(cuda_device, 61)
    u, Bm, Cm = r(1, T, D), r(1, T, 1, N), torch.zeros(1, T, 1, N, device=cuda_device)
    dy = torch.ones_like(u)
    u[0, 3::2, 2], dy[0, 3::2, 2] = 1e30, 1e30
    u[0, :, 5], dy[0, :, 5] = -3e38, 1.0
    g = gdr.scan_bwd(u, torch.full_like(u, 0.1), -torch.ones(D, N, device=cuda_device), Bm, Cm, torch.ones(D, device=cuda_device),
                     dy=dy)
    want = (u * dy).sum((0, 1))
    assert want[2] == INF and want[5] == -INF
    assert torch.equal(g["dD"].isinf(), want.isinf()) and g["dD"][2] == INF and g["dD"][5] == -INF
    assert torch.isfinite(g["dD"][[0, 1, 3, 4, 6, 7]]).all()


def test_scan_clears_the_rows_behind_a_short_sequence(cuda_device):
    """A block clears more than 2^31 places of its channel tile (T times 256)."""
    T, n = 9_000_000, 5
    r = Rnd(cuda_device, 51)
    u, Bm, Cm = r(1, T, 1, dtype=BF), r(1, T, 1, 1, dtype=BF), r(1, T, 1, 1, dtype=BF)
    A = torch.full((1, 1), -0.5, device=cuda_device)
    out = torch.full((1, T, 1), NAN, dtype=BF, device=cuda_device)
    lengths = torch.tensor([n], dtype=torch.int32, device=cuda_device)
    want, h = gdr.scan_fwd(u[:, :n], u[:, :n].abs(), A, Bm[:, :n], Cm[:, :n])
    y, h_T = gdr.scan_fwd(u, u.abs(), A, Bm, Cm, lengths=lengths, out=out, workspace=None)
    assert y is out and torch.equal(y[:, :n], want) and torch.equal(h_T, h)
    assert (y[:, n:] == 0).all()


# ---------------------------------------------------------------- convolution

@pytest.mark.parametrize("B,T,D", [(32, 256, 14208), (8, 32768, 16)])
def test_conv_parameter_gradients_of_long_sums(cuda_device, B, T, D):
    """dweight and dbias over many tokens in one thread's chunk, or over many chunks.
    Every term is 1 + 63 2^-23, which a sum of 128 terms and more loses at every
    addition: one sum over 256 terms is 60 2^-24 off. Adding n equal numbers to 0 one
    after the other costs at most (n + 1) / 2 roundings of the sum; sums of 64 terms,
    of 4 such sums, of 16 partials, and the result's rounding come to 32.5 + 2.5 +
    8.5 + 1."""
    v = 1 + 63 * 2.0 ** -23
    x, dy = (torch.full((1, 1, D), c, device=cuda_device).expand(B, T, D) for c in (1.0, v))
    w, b = torch.ones(D, 2, device=cuda_device), torch.zeros(D, device=cuda_device)
    g = gdr.conv_bwd(x, w, b, dy=dy, activation=None)
    for got, n in ((g["dweight"][:, 1], B * T), (g["dweight"][:, 0], B * (T - 1)), (g["dbias"], B * T)):
        off = ((got.double() - n * v).abs().max() / (n * v)).item()
        assert off <= 45 * R.U32, off / R.U32


@pytest.mark.parametrize("W,D", [(4, (1 << 29) + 2), (2, (1 << 30) + 1)])
def test_conv_of_a_very_wide_layer(cuda_device, W, D):
    """More than 2^31 filter taps: the first and last channels as in a layer of their own."""
    x = torch.randn(1, 1, D, device=cuda_device, dtype=BF)
    w = torch.randn(D, W, device=cuda_device, dtype=BF)
    y, X = gdr.conv_fwd(x, w)
    for s in (slice(0, 6), slice(D // 2, D // 2 + 6), slice(D - 5, D)):
        want, X_want = gdr.conv_fwd(x[..., s], w[s].clone())
        assert torch.equal(y[..., s], want) and torch.equal(X[..., s], X_want)
    del y, X
    one = torch.zeros(1, W - 1, D, device=cuda_device, dtype=BF)
    y = gdr.conv_step(x[:, 0], w, None, one)
    assert torch.equal(y[:, :6], gdr.conv_fwd(x[..., :6], w[:6].clone())[0][:, 0])


def test_axes_beyond_int_are_refused(cuda_device):
    """Heads, groups and states too: cut to 32 bits they would be 1 or 4."""
    n = (1 << 32) + 1
    q = torch.zeros(1, 1, 1, 1, device=cuda_device, dtype=BF)
    with pytest.raises(ValueError, match="k has an axis of 4294967297"):
        gdr.qk_norm_fwd(q, q.expand(1, 1, n, 1))
    u, A = torch.zeros(1, 1, 1, device=cuda_device, dtype=BF), torch.zeros(1, 1, device=cuda_device)
    with pytest.raises(ValueError, match="Bm has an axis of 4294967297"):
        wide = torch.empty(1, 1, n, 1, device=cuda_device, dtype=BF)
        gdr.scan_fwd(u, u, A, wide, wide)
    with pytest.raises(ValueError, match="A has an axis of 4294967297"):
        gdr.scan_fwd(u, u, torch.empty(1, n, device=cuda_device), wide.view(1, 1, 1, n), wide.view(1, 1, 1, n))


# ---------------------------------------------------------------- results in place

def test_in_place_refusals(cuda_device):
    """A result may be its own input, dense; no other input, the same tensor given
    twice included, and no other order of the rows."""
    r = Rnd(cuda_device, 41)
    buf = r(2, 3, 4, 16)
    q, k = buf.transpose(1, 2), r(2, 4, 3, 16)
    before = buf.clone()
    with pytest.raises(ValueError, match="q_out overlaps q"):
        gdr.qk_norm_fwd(q, k, q_out=buf.view(2, 4, 3, 16))
    with pytest.raises(ValueError, match="k_out overlaps k"):
        gdr.qk_norm_fwd(k, q, k_out=buf.view(2, 4, 3, 16))
    with pytest.raises(ValueError, match="q_out overlaps k"):
        gdr.qk_norm_fwd(buf, buf, q_out=buf)
    with pytest.raises(ValueError, match="k_out overlaps q"):
        gdr.qk_norm_fwd(buf, buf, k_out=buf)
    x = r(2, 3, 8)
    kept = x.clone()
    with pytest.raises(ValueError, match="X_T overlaps x"):
        gdr.conv_fwd(x, r(8, 4), None, x, X_T=x)
    s = r(1, 4, 4)
    with pytest.raises(ValueError, match="h_T overlaps u"):
        gdr.scan_fwd(s, s.clone(), -torch.ones(4, 4, device=cuda_device), r(1, 4, 1, 4), r(1, 4, 1, 4), None, None, s, h_T=s)
    torch.cuda.synchronize()
    assert torch.equal(buf, before) and torch.equal(x, kept)
    want, _ = gdr.qk_norm_fwd(buf)
    got, _ = gdr.qk_norm_fwd(buf, q_out=buf)
    assert got is buf and torch.equal(buf, want)


# ---------------------------------------------------------------- norm and rotation

@pytest.mark.parametrize("dtype,d,rot", [(BF, 256, 64), (F32, 72, 72), (BF, 114, 56)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_backward_of_more_tokens_than_one_turn(cuda_device, dtype, d, rot, layout):
    """More blocks of tokens than are launched: positions, turns and the weights' sums
    go on from one turn to the next (5103 tokens, 319 blocks of 16 or more of fewer;
    296 are launched), the last one partly filled."""
    B, T, Hq, Hk = 3, 1701, 2, 1
    r = Rnd(cuda_device, d)
    q, k, dq, dk = (r(B, T, H, d, dtype=dtype) for H in (Hq, Hk, Hq, Hk))
    qw, kw = r(d), r(d)
    f = torch.exp(-torch.arange(rot // 2) / 3.0).to(cuda_device)
    p = r.ints(-(1 << 20), 1 << 20, B, T)
    kws = dict(kind="rms", eps=1e-5, q_scale=0.5, positions=p, inv_freq=f, rotary=layout)
    g = gdr.qk_norm_bwd(q, k, qw, kw, dq=dq, dk=dk, **kws)
    for x, w, do, n, s, H in ((q, qw, dq, "q", 0.5, Hq), (k, kw, dk, "k", 1.0, Hk)):
        v, m = R.norm(x, w, "rms", 1e-5, s, p, f, layout, 1.0, do)
        R.check(g["d" + n], v["dx"], m["dx"], 100, "d" + n)
        R.check(g[f"d{n}_weight"], v["dw"], m["dw"], 100 + B * T * H, f"d{n}_weight")
