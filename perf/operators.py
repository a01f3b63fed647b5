"""Workloads of the operators that stand beside the gated delta-rule recurrence: the short causal
convolution, the selective state-space scan and the per-head norm of queries and keys.

Each case is one call as a program makes it. `run` computes it in plain torch operations (32 bits
inside, rounded once at the end) or, where `own` is true, with this package's kernels; `exact`
computes the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # q, k, v of 16 q/k heads and 32 value heads of width 128, convolved before the recurrence
        dict(name="conv-prompt", op="conv_fwd", dtype="bf16", B=2, T=4096, D=8192, W=4, bias=False,
             state=False, ragged=False, silu=True),
        # a padded batch of prompts of odd lengths that continue a cached prefix, fp32
        dict(name="conv-ragged", op="conv_fwd", dtype="fp32", B=5, T=1021, D=2056, W=3, bias=True,
             state=True, ragged=True, silu=True),
        # training step of the same layer at 16 heads: gradients of x, the filter, bias and state
        dict(name="conv-train", op="conv_bwd", dtype="bf16", B=4, T=4096, D=6144, W=4, bias=True,
             state=True, ragged=False, silu=True),
        # one token of 256 sequences, q, k, v of 32 heads
        dict(name="conv-decode", op="conv_step", dtype="bf16", B=256, T=1, D=12288, W=4, bias=True,
             state=True, ragged=False, silu=True),
        # a batch of prompts through the scan
        dict(name="scan-prompt", op="scan_fwd", dtype="bf16", B=4, T=4096, D=4096, N=16, G=1,
             state=False, ragged=False, gate=True, skip=True),
        # one long prompt that continues from a carried state: few channels, a long axis
        dict(name="scan-long", op="scan_fwd", dtype="bf16", B=1, T=32768, D=2048, N=16, G=1,
             state=True, ragged=False, gate=True, skip=True),
        # training step on a padded batch, two groups of input / output vectors
        dict(name="scan-train", op="scan_bwd", dtype="bf16", B=2, T=4096, D=4096, N=16, G=2,
             state=True, ragged=True, gate=True, skip=True),
        # one token of 256 sequences
        dict(name="scan-decode", op="scan_step", dtype="bf16", B=256, T=1, D=4096, N=16, G=1,
             state=True, ragged=False, gate=True, skip=True),
        # one token of one sequence: latency
        dict(name="scan-decode-one", op="scan_step", dtype="fp32", B=1, T=1, D=2048, N=16, G=1,
             state=True, ragged=False, gate=True, skip=True),
        # L2 norm and rotation of 32 + 32 heads before the recurrence
        dict(name="norm-prompt", op="qk_norm_fwd", dtype="bf16", B=2, T=8192, Hq=32, Hk=32, d=128,
             rot=128, rotary="half", kind="l2", weight=False, far=0),
        # training step at the 256-wide heads: root-mean-square norm with weights, part of the head rotated
        dict(name="norm-train", op="qk_norm_bwd", dtype="bf16", B=2, T=4096, Hq=16, Hk=16, d=256,
             rot=64, rotary="interleaved", kind="rms", weight=True, far=0),
        # one token of 256 sequences at far positions, grouped heads
        dict(name="norm-decode", op="qk_norm_fwd", dtype="bf16", B=256, T=1, Hq=32, Hk=8, d=128,
             rot=64, rotary="half", kind="rms", weight=True, far=1000000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step",
                     "qk_norm_fwd", "qk_norm_bwd"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op.startswith("conv"):
        step = op == "conv_step"
        B = _log(rng, 1, 256) if step else _log(rng, 1, 8)
        D = _log(rng, 16, 12288) if rng.random() < 0.4 else 8 * _log(rng, 4, 1536)
        T = 1 if step else _log(rng, 1, 32768)
        T = max(1, min(T, (32 << 20) // (B * D)))
        c.update(B=B, T=T, D=D, W=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.5,
                 state=step or rng.random() < 0.5, ragged=not step and rng.random() < 0.5,
                 silu=rng.random() < 0.75)
    elif op.startswith("scan"):
        step = op == "scan_step"
        B = _log(rng, 1, 256) if step else _log(rng, 1, 8)
        G = rng.choice([1, 1, 2, 4])
        D = G * (_log(rng, 16, 1024) if rng.random() < 0.5 else 16 * _log(rng, 2, 64))
        N = rng.choice([4, 8, 16, 16, 16, 24, 32, 64])
        T = 1 if step else _log(rng, 1, 32768)
        T = max(1, min(T, (256 << 20) // (B * D * N), 8192 if op == "scan_bwd" else 32768))
        c.update(B=B, T=T, D=D, N=N, G=G, state=step or rng.random() < 0.5,
                 ragged=not step and rng.random() < 0.5, gate=rng.random() < 0.7,
                 skip=rng.random() < 0.8)
    else:
        B, d = _log(rng, 1, 64), rng.choice([64, 128, 128, 256, 8 * _log(rng, 2, 32), _log(rng, 16, 256)])
        Hk = _log(rng, 1, 32)
        Hq = Hk * rng.choice([1, 1, 2, 4])
        T = _log(rng, 1, 8192)
        T = max(1, min(T, (48 << 20) // (B * (Hq + Hk) * d)))
        rot = rng.choice([0, d // 2 * 2, d // 4 * 2])
        kind = rng.choice(["l2", "rms"])
        c.update(B=B, T=T, Hq=Hq, Hk=Hk, d=d, rot=rot, rotary=rng.choice(["half", "interleaved"]),
                 kind=kind, weight=kind == "rms" and rng.random() < 0.8, far=rng.choice([0, 0, 100000, 1000000]))
    return c


def _esize(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    e, op, B, T = _esize(case), case["op"], case["B"], case["T"]
    if op.startswith("conv"):
        D, W = case["D"], case["W"]
        n = B * T * D
        state = B * (W - 1) * D * e
        act = 6 if case["silu"] else 0
        if op == "conv_fwd":
            return {"bytes": 2 * n * e + state * (1 + case["state"]) + D * W * e, "flops": n * (2 * W + act)}
        if op == "conv_step":
            return {"bytes": 2 * n * e + 2 * state + D * W * e, "flops": n * (2 * W + act)}
        return {"bytes": n * (2 * e + 4) + state * case["state"] + 2 * B * (W - 1) * D * 4 + D * W * (e + 4),
                "flops": n * (6 * W + 2 * act)}
    if op.startswith("scan"):
        D, N, G = case["D"], case["N"], case["G"]
        n, gates = B * T * D, int(case["gate"])
        state = B * D * N * 4
        bc = 2 * B * T * G * N
        if op == "scan_fwd":
            return {"bytes": n * e * (3 + gates) + bc * e + state * (1 + case["state"]) + D * N * 4,
                    "flops": n * (7 * N + 10)}
        if op == "scan_step":
            return {"bytes": n * e * (3 + gates) + bc * e + 2 * state + D * N * 4, "flops": n * (7 * N + 10)}
        return {"bytes": n * (e * (3 + gates) + 4 * (2 + gates)) + bc * (e + 4) + state * (2 + case["state"]) + 2 * D * N * 4,
                "flops": n * (24 * N + 30)}
    rows = B * T * (case["Hq"] + case["Hk"])
    n = rows * case["d"]
    if op == "qk_norm_fwd":
        return {"bytes": 2 * n * e, "flops": 4 * n + 3 * rows * case["rot"]}
    return {"bytes": n * (2 * e + 4), "flops": 10 * n + 3 * rows * case["rot"]}


# ---------------------------------------------------------------- inputs

def _lengths(case, g):
    if not case["ragged"]:
        return None
    n = torch.randint(max(1, case["T"] // 2), case["T"] + 1, (case["B"],), generator=g, device=DEV)
    n[0] = case["T"]
    return n.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt, B, T = DTYPES[case["dtype"]], case["B"], case["T"]

    def normal(*shape, scale=1.0, dtype=None):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype or dt)

    s = {"case": dict(case)}
    op = case["op"]
    if op.startswith("conv"):
        D, W = case["D"], case["W"]
        x = normal(B, T, D)
        s.update(x=x[:, 0] if op == "conv_step" else x, weight=normal(D, W, scale=W ** -0.5),
                 bias=normal(D, scale=0.1) if case["bias"] else None,
                 X=normal(B, W - 1, D) if case["state"] else None, lengths=_lengths(case, g))
        if op == "conv_bwd":
            s.update(dy=normal(B, T, D), dX_T=normal(B, W - 1, D, dtype=torch.float32))
    elif op.startswith("scan"):
        D, N, G = case["D"], case["N"], case["G"]
        # u beside its gate, and B, C beside the step's low-rank part, as projections leave them
        uz = normal(B, T, 2 * D)
        rank = max(8, D // 16 // 8 * 8)
        proj = normal(B, T, rank + 2 * G * N)
        step0 = torch.exp(torch.rand((D,), generator=g, device=DEV) * math.log(100.0) + math.log(1e-3))
        s.update(u=uz[..., :D].contiguous(), delta=normal(B, T, D, scale=0.5),
                 A=-torch.arange(1, N + 1, device=DEV, dtype=torch.float32)
                 * torch.exp(0.2 * torch.randn((D, N), generator=g, device=DEV)),
                 Bm=proj[..., rank:rank + G * N].view(B, T, G, N),
                 Cm=proj[..., rank + G * N:].view(B, T, G, N),
                 D=1 + 0.1 * torch.randn((D,), generator=g, device=DEV) if case["skip"] else None,
                 z=uz[..., D:] if case["gate"] else None,
                 delta_bias=step0 + torch.log(-torch.expm1(-step0)),
                 h=0.5 * torch.randn((B, D, N), generator=g, device=DEV) if case["state"] else None,
                 lengths=_lengths(case, g))
        if op == "scan_step":
            for k in ("u", "delta", "Bm", "Cm", "z"):
                if s[k] is not None:
                    s[k] = s[k][:, 0]
        if op == "scan_bwd":
            s.update(dy=normal(B, T, D), dh_T=torch.randn((B, D, N), generator=g, device=DEV))
    else:
        Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
        qkv = normal(B, T, (Hq + 2 * Hk) * d)  # v stands behind q and k
        s.update(q=qkv[..., :Hq * d].view(B, T, Hq, d), k=qkv[..., Hq * d:(Hq + Hk) * d].view(B, T, Hk, d),
                 q_weight=None, k_weight=None, positions=None, inv_freq=None)
        if case["weight"]:
            s.update(q_weight=1 + normal(d, scale=0.1), k_weight=1 + normal(d, scale=0.1))
        if case["rot"]:
            i = torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"]
            s["inv_freq"] = (10000.0 ** -i).float()
            start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device=DEV)
            s["positions"] = start + torch.arange(T, device=DEV)
        if op == "qk_norm_bwd":
            s.update(dq=normal(B, T, Hq, d), dk=normal(B, T, Hk, d))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    import gated_delta_rule_147_b200 as gdr

    c = s["case"]
    op = c["op"]
    if op.startswith("conv"):
        act = "silu" if c["silu"] else None
        if op == "conv_fwd":
            return gdr.conv_fwd(s["x"], s["weight"], s["bias"], s["X"], activation=act, lengths=s["lengths"])
        if op == "conv_bwd":
            return gdr.conv_bwd(s["x"], s["weight"], s["bias"], s["X"], dy=s["dy"], dX_T=s["dX_T"],
                                activation=act, lengths=s["lengths"], need_dX0=s["X"] is not None)
        y = gdr.conv_step(s["x"], s["weight"], s["bias"], s["X"], activation=act)
        return y, s["X"]
    if op.startswith("scan"):
        args = (s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"], s["h"])
        kw = dict(delta_bias=s["delta_bias"], delta_softplus=True)
        if op == "scan_fwd":
            return gdr.scan_fwd(*args, lengths=s["lengths"], **kw)
        if op == "scan_bwd":
            return gdr.scan_bwd(*args, dy=s["dy"], dh_T=s["dh_T"], lengths=s["lengths"],
                                need_dh0=s["h"] is not None, **kw)
        return gdr.scan_step(*args, **kw), s["h"]
    kw = dict(kind=c["kind"], eps=1e-6, q_scale=c["d"] ** -0.5, positions=s["positions"],
              inv_freq=s["inv_freq"], rotary=c["rotary"])
    if op == "qk_norm_fwd":
        return gdr.qk_norm_fwd(s["q"], s["k"], s["q_weight"], s["k_weight"], **kw)
    return gdr.qk_norm_bwd(s["q"], s["k"], s["q_weight"], s["k_weight"], dq=s["dq"], dk=s["dk"], **kw)


def _sig(x):
    return 1 / (1 + torch.exp(-x))


def _valid(s, T):
    """[B, T, 1] truth values of the tokens that a sequence has, or None where all have T."""
    if s["lengths"] is None:
        return None
    return (torch.arange(T, device=DEV)[None, :] < s["lengths"][:, None])[..., None]


def _mask(x, ok):
    return x if ok is None or x is None else torch.where(ok.view(ok.shape + (1,) * (x.dim() - 3)), x, 0)


def _conv_rows(s):
    """The inputs with the carried rows before them, in 32 bits, and the row each sequence ends at."""
    x, W = s["x"], s["weight"].shape[1]
    B, T, D = x.shape
    X = torch.zeros((B, W - 1, D), device=DEV) if s["X"] is None else s["X"].float()
    ext = torch.cat([X, _mask(x, _valid(s, T)).float()], 1)
    n = torch.full((B,), T, device=DEV) if s["lengths"] is None else s["lengths"].long()
    tail = n[:, None] + torch.arange(W - 1, device=DEV)
    return ext, tail


def _conv_pre(s, ext, T):
    w = s["weight"].float()
    p = w[:, 0] * ext[:, :T]
    for j in range(1, w.shape[1]):
        p = p + w[:, j] * ext[:, j:j + T]
    return p if s["bias"] is None else p + s["bias"].float()


def _plain_conv_fwd(s):
    x, T = s["x"], s["x"].shape[1]
    ext, tail = _conv_rows(s)
    p = _conv_pre(s, ext, T)
    y = p * _sig(p) if s["case"]["silu"] else p
    X_T = ext[torch.arange(x.shape[0], device=DEV)[:, None], tail]
    return _mask(y, _valid(s, T)).to(x.dtype), X_T.to(x.dtype)


def _plain_conv_bwd(s):
    x, w = s["x"], s["weight"].float()
    B, T, D = x.shape
    W = w.shape[1]
    ext, tail = _conv_rows(s)
    dp = _mask(s["dy"].float(), _valid(s, T))
    if s["case"]["silu"]:
        p = _conv_pre(s, ext, T)
        sg = _sig(p)
        dp = dp * (sg * (1 + p * (1 - sg)))
    dext = torch.zeros_like(ext)
    dext[torch.arange(B, device=DEV)[:, None], tail] = s["dX_T"]
    dw = torch.empty((D, W), device=DEV)
    for j in range(W):
        dext[:, j:j + T] += w[:, j] * dp
        dw[:, j] = (dp * ext[:, j:j + T]).sum((0, 1))
    return {"dx": dext[:, W - 1:].contiguous(), "dweight": dw,
            "dbias": None if s["bias"] is None else dp.sum((0, 1)),
            "dX0": None if s["X"] is None else dext[:, :W - 1].contiguous()}


def _plain_conv_step(s):
    ext = torch.cat([s["X"], s["x"][:, None]], 1).float()
    p = _conv_pre(s, ext, 1)[:, 0]
    y = p * _sig(p) if s["case"]["silu"] else p
    s["X"].copy_(ext[:, 1:])
    return y.to(s["x"].dtype), s["X"]


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


_BLOCK = 64


def _heads(m, D):
    """[B, t, G, N] vectors for each of D channels, in 32 bits."""
    B, t, G, N = m.shape
    return m.float()[:, :, :, None, :].expand(B, t, G, D // G, N).reshape(B, t, D, N)


def _scan_states(s, u, dt, Bm, h, keep):
    """Steps h through the tokens; returns the last state and, for each block of tokens, what `keep`
    makes of the block's decays and states."""
    T, D = u.shape[1:]
    A, got = s["A"], []
    for t0 in range(0, T, _BLOCK):
        t1 = min(T, t0 + _BLOCK)
        a = torch.exp(dt[:, t0:t1, :, None] * A)
        hs = (dt[:, t0:t1] * u[:, t0:t1])[..., None] * _heads(Bm[:, t0:t1], D)
        for i in range(t1 - t0):
            torch.addcmul(hs[:, i], a[:, i], h, out=hs[:, i])
            h = hs[:, i]
        got.append(keep(t0, t1, hs))
        h = h.clone()
    return h, got


def _scan_inputs(s):
    ok = _valid(s, s["u"].shape[1])
    raw = s["delta"].float() + s["delta_bias"]
    dt = _mask(_softplus(raw), ok)
    return ok, raw, _mask(s["u"].float(), ok), dt, _mask(s["Bm"], ok), _mask(s["Cm"], ok)


def _state0(s):
    B, D = s["u"].shape[0], s["u"].shape[-1]
    return torch.zeros((B, D, s["A"].shape[1]), device=DEV) if s["h"] is None else s["h"].clone()


def _plain_scan_fwd(s):
    D = s["u"].shape[-1]
    ok, _, u, dt, Bm, Cm = _scan_inputs(s)
    h, y = _scan_states(s, u, dt, Bm, _state0(s), lambda t0, t1, hs: (hs * _heads(Cm[:, t0:t1], D)).sum(-1))
    y = torch.cat(y, 1)
    if s["D"] is not None:
        y = y + s["D"] * u
    if s["z"] is not None:
        z = _mask(s["z"].float(), ok)
        y = y * (z * _sig(z))
    return _mask(y, ok).to(s["u"].dtype), h


def _plain_scan_bwd(s):
    B, T, D = s["u"].shape
    A, G = s["A"], s["Bm"].shape[2]
    N = A.shape[1]
    ok, raw, u, dt, Bm, Cm = _scan_inputs(s)
    h0 = _state0(s)
    _, hs = _scan_states(s, u, dt, Bm, h0, lambda t0, t1, hs: hs)
    dy, z = _mask(s["dy"].float(), ok), s["z"]
    if z is not None:
        z = _mask(z.float(), ok)
        sg = _sig(z)
        gate, dy_out = z * sg, dy
        dy = dy * gate
    f32 = dict(device=DEV, dtype=torch.float32)
    du, ddt, yh = torch.empty((B, T, D), **f32), torch.empty((B, T, D), **f32), torch.empty((B, T, D), **f32)
    dB, dC = torch.empty((B, T, G, N), **f32), torch.empty((B, T, G, N), **f32)
    dA = torch.zeros((D, N), **f32)
    g = s["dh_T"].clone()
    for blk in range(len(hs) - 1, -1, -1):
        t0 = blk * _BLOCK
        t1 = min(T, t0 + _BLOCK)
        h = hs[blk]
        hs[blk] = None
        a = torch.exp(dt[:, t0:t1, :, None] * A)
        before = hs[blk - 1][:, -1:] if blk else h0[:, None]
        Bx, Cx = _heads(Bm[:, t0:t1], D), _heads(Cm[:, t0:t1], D)
        gs = dy[:, t0:t1, :, None] * Cx
        for i in range(t1 - t0 - 1, -1, -1):
            gs[:, i] += g
            g = a[:, i] * gs[:, i]
        yh[:, t0:t1] = (h * Cx).sum(-1)
        dC[:, t0:t1] = (dy[:, t0:t1, :, None] * h).view(B, t1 - t0, G, D // G, N).sum(3)
        dB[:, t0:t1] = (gs * (dt * u)[:, t0:t1, :, None]).view(B, t1 - t0, G, D // G, N).sum(3)
        gB = (gs * Bx).sum(-1)
        du[:, t0:t1] = gB * dt[:, t0:t1]
        ah = gs * a * torch.cat([before, h[:, :-1]], 1)
        ddt[:, t0:t1] = gB * u[:, t0:t1] + (ah * A).sum(-1)
        dA += (ah * dt[:, t0:t1, :, None]).sum((0, 1))
    out = {"dA": dA, "dB": dB, "dC": dC, "dh0": None if s["h"] is None else g, "dD": None, "dz": None}
    if s["D"] is not None:
        out["dD"] = (dy * u).sum((0, 1))
        du = du + s["D"] * dy
        yh = yh + s["D"] * u
    if z is not None:
        out["dz"] = dy_out * yh * (sg * (1 + z * (1 - sg)))
    ddelta = _mask(ddt * _sig(raw), ok)
    out.update(du=_mask(du, ok), ddelta=ddelta, ddelta_bias=ddelta.sum((0, 1)))
    return out


def _plain_scan_step(s):
    u = s["u"].float()
    D = u.shape[-1]
    dt = _softplus(s["delta"].float() + s["delta_bias"])
    h = torch.exp(dt[..., None] * s["A"]) * s["h"] + (dt * u)[..., None] * _heads(s["Bm"][:, None], D)[:, 0]
    y = (h * _heads(s["Cm"][:, None], D)[:, 0]).sum(-1)
    if s["D"] is not None:
        y = y + s["D"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * _sig(z))
    s["h"].copy_(h)
    return y.to(s["u"].dtype), s["h"]


def _turn(s):
    """Cosines and sines [B, T, 1, rot / 2]; the angles of far positions in 64 bits."""
    ang = s["positions"].double()[..., None, None] * s["inv_freq"].double()
    return torch.cos(ang).float(), torch.sin(ang).float()


def _rotate(s, x, back=False):
    c = s["case"]
    r = c["rot"]
    if not r:
        return x
    cos, sin = _turn(s)
    sin = -sin if back else sin
    i = torch.arange(r // 2, device=DEV)
    first, second = (i, i + r // 2) if c["rotary"] == "half" else (2 * i, 2 * i + 1)
    x1, x2 = x[..., first], x[..., second]
    out = x.clone()
    out[..., first] = x1 * cos - x2 * sin
    out[..., second] = x2 * cos + x1 * sin
    return out


def _norm(s, x, w):
    ss = (x * x).sum(-1, keepdim=True)
    if s["case"]["kind"] == "l2":
        return x / torch.clamp(torch.sqrt(ss), min=1e-6)
    x = x / torch.sqrt(ss / x.shape[-1] + 1e-6)
    return x if w is None else x * w.float()


def _plain_norm_fwd(s):
    scale = s["case"]["d"] ** -0.5
    q = _rotate(s, _norm(s, s["q"].float(), s["q_weight"])) * scale
    k = _rotate(s, _norm(s, s["k"].float(), s["k_weight"]))
    return q.to(s["q"].dtype), k.to(s["k"].dtype)


def _plain_norm_bwd(s):
    c, out = s["case"], {}
    for n, scale in (("q", c["d"] ** -0.5), ("k", 1.0)):
        x, w = s[n].float(), s[n + "_weight"]
        g = _rotate(s, s["d" + n].float() * scale, back=True)
        ss = (x * x).sum(-1, keepdim=True)
        if c["kind"] == "l2":
            r = 1 / torch.clamp(torch.sqrt(ss), min=1e-6)
            xh = x * r
            dx = torch.where(torch.sqrt(ss) > 1e-6, r * (g - xh * (g * xh).sum(-1, keepdim=True)), r * g)
            dw = None
        else:
            r = 1 / torch.sqrt(ss / c["d"] + 1e-6)
            xh = x * r
            dw = None if w is None else (g * xh).sum((0, 1, 2))
            gw = g if w is None else g * w.float()
            dx = r * (gw - xh * ((gw * xh).sum(-1, keepdim=True) / c["d"]))
        out["d" + n] = dx
        out["d" + n + "_weight"] = dw
    return out


_PLAIN = {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
          "scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step,
          "qk_norm_fwd": _plain_norm_fwd, "qk_norm_bwd": _plain_norm_bwd}


# ---------------------------------------------------------------- the definitions in 64 bits

def _f64(v):
    return None if v is None else v.double()


def _silu64(p):
    """silu and its derivative."""
    e = torch.special.expit(p)
    return p * e, e + p * e * (1 - e)


def _exact_conv(s):
    """One sequence at a time, from its own rows only."""
    c, op = s["case"], s["case"]["op"]
    x = s["x"][:, None] if op == "conv_step" else s["x"]
    B, T, D = x.shape
    w, bias = _f64(s["weight"]), _f64(s["bias"])
    W = w.shape[1]
    f64 = dict(dtype=torch.float64, device=DEV)
    y, X_T = torch.zeros((B, T, D), **f64), torch.zeros((B, W - 1, D), **f64)
    dx, dX0 = torch.zeros((B, T, D), **f64), torch.zeros((B, W - 1, D), **f64)
    dw, db = torch.zeros((D, W), **f64), torch.zeros((D,), **f64)
    for b in range(B):
        n = T if s["lengths"] is None else int(s["lengths"][b])
        before = torch.zeros((W - 1, D), **f64) if s["X"] is None else s["X"][b].double()
        rows = torch.cat([before, x[b, :n].double()])
        p = torch.stack([rows[j:j + n] for j in range(W)], -1).mul_(w).sum(-1)
        p = p if bias is None else p + bias
        f, df = _silu64(p) if c["silu"] else (p, torch.ones_like(p))
        y[b, :n], X_T[b] = f, rows[n:]
        if op == "conv_bwd":
            dp = s["dy"][b, :n].double() * df
            drows = torch.cat([torch.zeros((n, D), **f64), s["dX_T"][b].double()])
            for j in range(W):
                drows[j:j + n] += dp * w[:, j]
                dw[:, j] += torch.einsum("td,td->d", dp, rows[j:j + n])
            db += dp.sum(0)
            dX0[b], dx[b, :n] = drows[:W - 1], drows[W - 1:]
    if op == "conv_bwd":
        return {"dx": dx, "dweight": dw, "dbias": None if bias is None else db,
                "dX0": None if s["X"] is None else dX0}
    return (y[:, 0] if op == "conv_step" else y), X_T


def _exact_scan(s):
    """Token by token, the channels as [groups, channels of a group]."""
    op = s["case"]["op"]
    step = op == "scan_step"
    grow = (lambda v: None if v is None else v[:, None].double()) if step else _f64
    u, raw, Bm, Cm, z = (grow(s[k]) for k in ("u", "delta", "Bm", "Cm", "z"))
    B, T, D = u.shape
    G, N = Bm.shape[2:]
    K = D // G
    raw = raw + _f64(s["delta_bias"])
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    on = torch.ones((B, T, 1), dtype=torch.float64, device=DEV)
    if s["lengths"] is not None:
        on = (torch.arange(T, device=DEV)[None] < s["lengths"][:, None]).double()[..., None]
    u, dt = u * on, dt * on
    A, f64 = _f64(s["A"]).view(G, K, N), dict(dtype=torch.float64, device=DEV)
    h = torch.zeros((B, G, K, N), **f64) if s["h"] is None else _f64(s["h"]).reshape(B, G, K, N)
    u4, dt4 = u.view(B, T, G, K), dt.view(B, T, G, K)
    yh = torch.empty((B, T, D), **f64)
    back = op == "scan_bwd"
    hist = [h]
    for t in range(T):
        h = torch.exp(dt4[:, t, ..., None] * A) * h
        h = h + torch.einsum("bgk,bgn->bgkn", dt4[:, t] * u4[:, t], Bm[:, t])
        yh[:, t] = torch.einsum("bgkn,bgn->bgk", h, Cm[:, t]).reshape(B, D)
        if back:
            hist.append(h)
    if s["D"] is not None:
        yh = yh + _f64(s["D"]) * u
    f, df = (torch.ones_like(yh), torch.zeros_like(yh)) if z is None else _silu64(z)
    if not back:
        y = yh * f * on
        return (y[:, 0] if step else y), h.reshape(B, D, N)
    dout = _f64(s["dy"]) * on
    dyh = dout * f
    d4 = dyh.view(B, T, G, K)
    du, ddt = torch.empty((B, T, G, K), **f64), torch.empty((B, T, G, K), **f64)
    dB, dC = torch.empty((B, T, G, N), **f64), torch.empty((B, T, G, N), **f64)
    dA = torch.zeros((G, K, N), **f64)
    g = _f64(s["dh_T"]).reshape(B, G, K, N)
    for t in range(T - 1, -1, -1):
        g = g + torch.einsum("bgk,bgn->bgkn", d4[:, t], Cm[:, t])
        dC[:, t] = torch.einsum("bgk,bgkn->bgn", d4[:, t], hist.pop())
        dB[:, t] = torch.einsum("bgkn,bgk->bgn", g, dt4[:, t] * u4[:, t])
        into = torch.einsum("bgkn,bgn->bgk", g, Bm[:, t])
        g = g * torch.exp(dt4[:, t, ..., None] * A)
        via = g * hist[-1]
        du[:, t] = into * dt4[:, t]
        ddt[:, t] = into * u4[:, t] + (via * A).sum(-1)
        dA += torch.einsum("bgkn,bgk->gkn", via, dt4[:, t])
    du = du.reshape(B, T, D)
    ddelta = ddt.reshape(B, T, D) * torch.special.expit(raw) * on
    if s["D"] is not None:
        du = du + dyh * _f64(s["D"])
    return {"du": du * on, "ddelta": ddelta, "dA": dA.reshape(D, N), "dB": dB, "dC": dC,
            "dD": None if s["D"] is None else torch.einsum("btd,btd->d", dyh, u),
            "dz": None if z is None else dout * yh * df, "ddelta_bias": ddelta.sum((0, 1)),
            "dh0": None if s["h"] is None else g.reshape(B, D, N)}


def _exact_norm(s):
    """The rotation as a product of complex numbers; gradients by the chain rule of x / r(x)."""
    c = s["case"]
    d, rot = c["d"], c["rot"]
    unit = None
    if rot:
        ang = s["positions"].double()[..., None] * s["inv_freq"].double()
        unit = torch.polar(torch.ones_like(ang), ang)[:, :, None]

    def turn(x, w):
        if w is None:
            return x
        head, tail = x[..., :rot], x[..., rot:]
        if c["rotary"] == "half":
            y = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * w
            return torch.cat([y.real, y.imag, tail], -1)
        y = torch.view_as_complex(head.reshape(head.shape[:-1] + (rot // 2, 2)).contiguous()) * w
        return torch.cat([torch.view_as_real(y).flatten(-2), tail], -1)

    res = {}
    for n, scale in (("q", d ** -0.5), ("k", 1.0)):
        x, w = s[n].double(), _f64(s[n + "_weight"])
        if c["kind"] == "l2":
            r = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
            small = r <= 1e-6
            r = torch.where(small, torch.full_like(r, 1e-6), r)
            dr = torch.where(small, torch.zeros_like(x), x / r)  # dr / dx
        else:
            r = torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)
            dr = x / (d * r)
        if c["op"] == "qk_norm_fwd":
            y = x / r
            res[n] = turn(y if w is None else y * w, unit) * scale
            continue
        g = turn(s["d" + n].double() * scale, None if unit is None else unit.conj())
        res["d" + n + "_weight"] = None if w is None else (g * (x / r)).sum((0, 1, 2))
        g = g if w is None else g * w
        res["d" + n] = g / r - (g * x).sum(-1, keepdim=True) / r ** 2 * dr
    return (res["q"], res["k"]) if c["op"] == "qk_norm_fwd" else res


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return (_exact_conv if op.startswith("conv") else _exact_scan if op.startswith("scan") else _exact_norm)(s)
