"""The operators around the recurrence: short causal convolution, norm of
queries and keys with the position rotation, and the selective state-space scan.

  conv_fwd / conv_bwd / conv_step   depthwise convolution of 2 to 4 taps
  qk_norm_fwd / qk_norm_bwd         per-head L2 or RMS norm and rotation
  scan_fwd / scan_bwd / scan_step   h = exp(dt A) h + dt u B, y = C h + D u

Activations may be slices of wider tensors (outer axes of any stride, the
innermost dense); results are new dense tensors, or go into `out=`. Gradients
are float32. `lengths` (int32 [B]) gives the tokens of each sequence of a
padded batch: rows behind them are not read, and results there are 0. Every
call runs on the tensors' device and, unless `stream` is given, on its current
stream. With `stream`, results are allocated on that stream and marked as used
by the current one; ordering the two streams is the caller's part. include/gdr.h
has the formulas and limits.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import (ACT_NONE, ACT_SILU, GDR_BF16, GDR_FP32, NORM_L2, NORM_RMS, ROTARY_HALF,
                   ROTARY_INTERLEAVED)

_CODE = {torch.bfloat16: GDR_BF16, torch.float32: GDR_FP32}
_ACT = {None: ACT_NONE, "none": ACT_NONE, "silu": ACT_SILU}
_NORM = {"l2": NORM_L2, "rms": NORM_RMS}
_ROTARY = {"half": ROTARY_HALF, "interleaved": ROTARY_INTERLEAVED}


def _first(name, t, ndim):
    """Type code and device of the tensor the others are held to."""
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32")
    if not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}; the library takes CUDA tensors")
    if t.dim() != ndim:
        raise ValueError(f"{name} has {t.dim()} axes; expected {ndim}")
    return code, t.device


def _check(name, t, shape, dtypes, dev, tail=1):
    """Shape, type and device; the last `tail` axes dense. Returns t's strides."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}; expected {' or '.join(str(d) for d in dtypes)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}; expected {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    st, want = t.stride(), 1
    for i in range(1, tail + 1):
        if shape[-i] > 1 and st[-i] != want:
            raise ValueError(f"{name}: the last {tail} axes must be dense" if tail > 1
                             else f"{name}: the innermost axis must be dense")
        want *= shape[-i]
    return st


def _dense(name, t, shape, dtypes, dev):
    if t is not None:
        _check(name, t, shape, dtypes, dev, 0)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _lengths(t, B, dev):
    if t is not None:
        _dense("lengths", t, (B,), (torch.int32,), dev)


def _span(t):
    """First and last byte address (exclusive) that t's elements lie in."""
    n = sum((s - 1) * st for s, st in zip(t.shape, t.stride())) + 1 if t.numel() else 0
    return t.data_ptr(), t.data_ptr() + n * t.element_size()


def _apart(name, t, others, same=None):
    """A given result t shares no memory with the (name, tensor) of `others`;
    `same` may be t's own memory, whole."""
    if t is None or not t.numel():
        return
    a0, a1 = _span(t)
    for other, o in others:
        if o is None or not o.numel() or (o is same and o.data_ptr() == a0 and o.is_contiguous()):
            continue
        b0, b1 = _span(o)
        if a0 < b1 and b0 < a1:
            raise ValueError(f"{name} overlaps {other}")


def _i64(*vals):
    return (ctypes.c_longlong * len(vals))(*vals)


class _Where:
    """The device and stream of one call. Tensors that the call makes come from
    the launch stream's pool, so nothing else can be using their memory."""

    def __init__(self, dev, stream):
        self.dev = dev
        self.side = None
        if stream is None:
            self.handle = torch.cuda.current_stream(dev).cuda_stream
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, dev) if stream else torch.cuda.default_stream(dev)
        elif stream.device != dev:
            raise ValueError(f"stream is on {stream.device}; expected {dev}")
        self.handle = stream.cuda_stream
        here = torch.cuda.current_stream(dev)
        if here.cuda_stream != self.handle:
            self.side, self.here = stream, here

    def empty(self, shape, dtype, result=True):
        if self.side is None:
            return torch.empty(shape, dtype=dtype, device=self.dev)
        with torch.cuda.stream(self.side):
            t = torch.empty(shape, dtype=dtype, device=self.dev)
        if result:
            t.record_stream(self.here)
        return t

    def scratch(self, given, nbytes):
        """(workspace, bytes): the caller's, or one of `nbytes` from torch."""
        if given is None:
            return self.empty(max(nbytes, 1), torch.uint8, result=False), max(nbytes, 1)
        if given.device != self.dev:
            raise ValueError(f"workspace is on {given.device}; expected {self.dev}")
        if not given.is_contiguous():
            raise ValueError("workspace must be contiguous")
        return given, given.numel() * given.element_size()

    def run(self, fn, *args):
        if torch.cuda.current_device() == self.dev.index:
            fn(*args, stream=self.handle)
        else:
            with torch.cuda.device(self.dev):
                fn(*args, stream=self.handle)


# ---------------------------------------------------------------- convolution

def _conv_params(x, weight, bias, dev, activation):
    D = x.shape[-1]
    if weight.dim() != 2:
        raise ValueError(f"weight has {weight.dim()} axes; expected 2")
    W = weight.shape[1]
    _dense("weight", weight, (D, W), (x.dtype, torch.float32), dev)
    _dense("bias", bias, (D,), (weight.dtype,), dev)
    if activation not in _ACT:
        raise ValueError(f"activation {activation!r}; expected 'silu' or None")
    return W, _ACT[activation], _CODE[weight.dtype]


def conv_fwd(x, weight, bias=None, X0=None, *, activation="silu", lengths=None, out=None,
             final_state=True, X_T=None, stream=None):
    """Short causal depthwise convolution over [B, T, D] inputs: weight [D, W],
    bias [D] (x's dtype or float32), X0 [B, W-1, D] the inputs before the first
    token (None: zeros), activation "silu" or None. Returns (y, X_T), X_T the
    last W - 1 inputs (None when final_state is False); X_T may be X0."""
    code, dev = _first("x", x, 3)
    B, T, D = x.shape
    W, act, wcode = _conv_params(x, weight, bias, dev, activation)
    own = (x.dtype,)
    sx = _check("x", x, (B, T, D), own, dev)
    for name, t, shape in (("X0", X0, (B, W - 1, D)), ("X_T", X_T, (B, W - 1, D)), ("out", out, (B, T, D))):
        _dense(name, t, shape, own, dev)
    _lengths(lengths, B, dev)
    ins = (("x", x), ("weight", weight), ("bias", bias), ("lengths", lengths), ("X0", X0))
    _apart("out", out, ins + (("X_T", X_T),))
    _apart("X_T", X_T, ins, X0)
    at = _Where(dev, stream)
    y = at.empty((B, T, D), x.dtype) if out is None else out
    if not final_state:
        X_T = None
    elif X_T is None:
        X_T = at.empty((B, W - 1, D), x.dtype)
    at.run(_lib.gdr_conv_fwd, x, weight, bias, X0, lengths, y, X_T, _i64(sx[0], sx[1]), B, T, D, W, act, code, wcode)
    return y, X_T


def conv_bwd(x, weight, bias=None, X0=None, *, dy, dX_T=None, activation="silu", lengths=None,
             workspace=None, need_dX0=True, stream=None):
    """Backward of conv_fwd for the same inputs: dy [B, T, D] in x's dtype or
    float32, dX_T [B, W-1, D] float32 or None. Returns a dict with dx, dweight,
    dbias (None without bias) and dX0 (None without X0 or need_dX0)."""
    code, dev = _first("x", x, 3)
    B, T, D = x.shape
    W, act, wcode = _conv_params(x, weight, bias, dev, activation)
    sx = _check("x", x, (B, T, D), (x.dtype,), dev)
    sg = _check("dy", dy, (B, T, D), (x.dtype, torch.float32), dev)
    _dense("X0", X0, (B, W - 1, D), (x.dtype,), dev)
    _dense("dX_T", dX_T, (B, W - 1, D), (torch.float32,), dev)
    _lengths(lengths, B, dev)
    at, f32 = _Where(dev, stream), torch.float32
    g = {"dx": at.empty((B, T, D), f32), "dweight": at.empty((D, W), f32),
         "dbias": None if bias is None else at.empty((D,), f32),
         "dX0": at.empty((B, W - 1, D), f32) if X0 is not None and need_dX0 else None}
    ws, nbytes = at.scratch(workspace, _lib.gdr_conv_bwd_workspace_size(B, T, D, W))
    at.run(_lib.gdr_conv_bwd, x, weight, bias, X0, lengths, dy, dX_T, g["dx"], g["dweight"], g["dbias"], g["dX0"],
           ws, nbytes, _i64(sx[0], sx[1], sg[0], sg[1]), B, T, D, W, act, code, wcode, _CODE[dy.dtype])
    return g


def conv_step(x, weight, bias, X, *, activation="silu", out=None, stream=None):
    """One token per sequence: x [B, D], X [B, W-1, D] the last inputs, moved on
    in place. Returns y [B, D]."""
    code, dev = _first("x", x, 2)
    B, D = x.shape
    W, act, wcode = _conv_params(x, weight, bias, dev, activation)
    own = (x.dtype,)
    sx = _check("x", x, (B, D), own, dev)
    _dense("X", X, (B, W - 1, D), own, dev)
    _dense("out", out, (B, D), own, dev)
    _apart("out", out, (("x", x), ("weight", weight), ("bias", bias), ("X", X)))
    at = _Where(dev, stream)
    y = at.empty((B, D), x.dtype) if out is None else out
    at.run(_lib.gdr_conv_step, x, weight, bias, X, y, _i64(sx[0]), B, D, W, act, code, wcode)
    return y


# ---------------------------------------------------------------- selective scan

def _scan_params(u, A, Bm, D, delta_bias, h, hname, lead, dev):
    f32 = (torch.float32,)
    if A.dim() != 2:
        raise ValueError(f"A has {A.dim()} axes; expected 2")
    if Bm.dim() != len(lead) + 2:
        raise ValueError(f"Bm has {Bm.dim()} axes; expected {len(lead) + 2}")
    Dn, N, G = u.shape[-1], A.shape[1], Bm.shape[-2]
    _dense("A", A, (Dn, N), f32, dev)
    _dense("D", D, (Dn,), f32, dev)
    _dense("delta_bias", delta_bias, (Dn,), f32, dev)
    _dense(hname, h, (lead[0], Dn, N), f32, dev)
    return Dn, N, G


def _scan_strides(u, delta, Bm, Cm, z, lead, Dn, N, G, dev, n):
    """Strides of the first n axes of u, delta, Bm, Cm, z."""
    own, st = (u.dtype,), []
    for name, t, shape, tail in (("u", u, lead + (Dn,), 1), ("delta", delta, lead + (Dn,), 1),
                                 ("Bm", Bm, lead + (G, N), 2), ("Cm", Cm, lead + (G, N), 2),
                                 ("z", z, lead + (Dn,), 1)):
        st += (0,) * n if t is None else _check(name, t, shape, own, dev, tail)[:n]
    return st


def scan_fwd(u, delta, A, Bm, Cm, D=None, z=None, h0=None, *, delta_bias=None, delta_softplus=False,
             lengths=None, workspace="auto", out=None, final_state=True, h_T=None, stream=None):
    """Selective scan over [B, T, D] inputs u and step sizes delta (delta_bias
    [D] added, then softplus with delta_softplus): A [D, N] and D [D] float32,
    Bm, Cm [B, T, G, N] shared by the D / G channels of a group, z [B, T, D] a
    gate (y z sigmoid(z)), h0 [B, D, N] float32 (None: zeros). Returns (y, h_T),
    h_T None when final_state is False; h_T may be h0. workspace: "auto" takes
    from torch what a split of the tokens needs (few channels, many tokens), a
    device tensor supplies it, None leaves the tokens unsplit."""
    code, dev = _first("u", u, 3)
    lead = tuple(u.shape[:2])
    B, T = lead
    Dn, N, G = _scan_params(u, A, Bm, D, delta_bias, h0, "h0", lead, dev)
    st = _scan_strides(u, delta, Bm, Cm, z, lead, Dn, N, G, dev, 2)
    _dense("h_T", h_T, (B, Dn, N), (torch.float32,), dev)
    _dense("out", out, lead + (Dn,), (u.dtype,), dev)
    _lengths(lengths, B, dev)
    if out is not None or h_T is not None:
        ins = (("u", u), ("delta", delta), ("A", A), ("Bm", Bm), ("Cm", Cm), ("D", D), ("z", z), ("h0", h0),
               ("delta_bias", delta_bias), ("lengths", lengths))
        _apart("out", out, ins + (("h_T", h_T),))
        _apart("h_T", h_T, ins, h0)
    at = _Where(dev, stream)
    y = at.empty(lead + (Dn,), u.dtype) if out is None else out
    if not final_state:
        h_T = None
    elif h_T is None:
        h_T = at.empty((B, Dn, N), torch.float32)
    ws, nbytes = None, 0
    if workspace is not None:
        nbytes = _lib.gdr_scan_fwd_workspace_size(B, T, Dn, N, G)
        if isinstance(workspace, str):
            if workspace != "auto":
                raise ValueError(workspace)
            workspace = None
        if nbytes:
            ws, nbytes = at.scratch(workspace, nbytes)
    at.run(_lib.gdr_scan_fwd, u, delta, A, Bm, Cm, D, z, delta_bias, h0, lengths, y, h_T, ws, nbytes, _i64(*st), B, T, Dn, N, G,
           int(bool(delta_softplus)), code)
    return y, h_T


def scan_bwd(u, delta, A, Bm, Cm, D=None, z=None, h0=None, *, dy, dh_T=None, delta_bias=None,
             delta_softplus=False, lengths=None, workspace=None, need_dh0=True, stream=None):
    """Backward of scan_fwd for the same inputs: dy [B, T, D] in u's dtype or
    float32, dh_T [B, D, N] float32 or None. Returns a dict with du, ddelta, dA,
    dB, dC, dD, dz, ddelta_bias and dh0 (None for what was absent, dh0 also
    without need_dh0)."""
    code, dev = _first("u", u, 3)
    lead = tuple(u.shape[:2])
    B, T = lead
    Dn, N, G = _scan_params(u, A, Bm, D, delta_bias, h0, "h0", lead, dev)
    st = _scan_strides(u, delta, Bm, Cm, z, lead, Dn, N, G, dev, 2)
    st += _check("dy", dy, lead + (Dn,), (u.dtype, torch.float32), dev)[:2]
    _dense("dh_T", dh_T, (B, Dn, N), (torch.float32,), dev)
    _lengths(lengths, B, dev)
    at, f32 = _Where(dev, stream), torch.float32
    g = {"du": at.empty(lead + (Dn,), f32), "ddelta": at.empty(lead + (Dn,), f32), "dA": at.empty((Dn, N), f32),
         "dB": at.empty(lead + (G, N), f32), "dC": at.empty(lead + (G, N), f32),
         "dD": None if D is None else at.empty((Dn,), f32),
         "dz": None if z is None else at.empty(lead + (Dn,), f32),
         "ddelta_bias": None if delta_bias is None else at.empty((Dn,), f32),
         "dh0": at.empty((B, Dn, N), f32) if h0 is not None and need_dh0 else None}
    ws, nbytes = at.scratch(workspace, _lib.gdr_scan_bwd_workspace_size(B, T, Dn, N, G))
    at.run(_lib.gdr_scan_bwd, u, delta, A, Bm, Cm, D, z, delta_bias, h0, lengths, dy, dh_T, g["du"], g["ddelta"],
           g["dA"], g["dB"], g["dC"], g["dD"], g["dz"], g["ddelta_bias"], g["dh0"], ws, nbytes, _i64(*st), B, T, Dn, N,
           G, int(bool(delta_softplus)), code, _CODE[dy.dtype])
    return g


def scan_step(u, delta, A, Bm, Cm, D, z, h, *, delta_bias=None, delta_softplus=False, out=None,
              stream=None):
    """One token per sequence: u, delta, z [B, D], Bm, Cm [B, G, N], h [B, D, N]
    float32 updated in place. Returns y [B, D]."""
    code, dev = _first("u", u, 2)
    lead = (u.shape[0],)
    Dn, N, G = _scan_params(u, A, Bm, D, delta_bias, h, "h", lead, dev)
    st = _scan_strides(u, delta, Bm, Cm, z, lead, Dn, N, G, dev, 1)
    _dense("out", out, lead + (Dn,), (u.dtype,), dev)
    _apart("out", out, (("u", u), ("delta", delta), ("A", A), ("Bm", Bm), ("Cm", Cm), ("D", D), ("z", z), ("h", h),
                        ("delta_bias", delta_bias)))
    at = _Where(dev, stream)
    y = at.empty(lead + (Dn,), u.dtype) if out is None else out
    at.run(_lib.gdr_scan_step, u, delta, A, Bm, Cm, D, z, delta_bias, h, y, _i64(*st), lead[0], Dn, N, G,
           int(bool(delta_softplus)), code)
    return y


# ---------------------------------------------------------------- norm and rotation

def _norm_params(q, k, q_weight, k_weight, kind, positions, inv_freq, rotary, dev):
    B, T, Hq, d = q.shape
    Hk = 0
    st = list(_check("q", q, (B, T, Hq, d), (q.dtype,), dev)[:3])
    if k is None:
        st += [0, 0, 0]
    else:
        if k.dim() != 4:
            raise ValueError(f"k has {k.dim()} axes; expected 4")
        Hk = k.shape[2]
        st += _check("k", k, (B, T, Hk, d), (q.dtype,), dev)[:3]
    wt = None
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _dense(name, w, (d,), (q.dtype, torch.float32) if wt is None else (wt,), dev)
            wt = w.dtype
    if kind not in _NORM:
        raise ValueError(f"kind {kind!r}; expected 'l2' or 'rms'")
    if rotary not in _ROTARY:
        raise ValueError(f"rotary {rotary!r}; expected 'half' or 'interleaved'")
    rot = pos64 = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        _dense("inv_freq", inv_freq, (rot // 2,), (torch.float32,), dev)
    if positions is not None:
        ps = _check("positions", positions, (B, T), (torch.int32, torch.int64), dev, 0)
        pos64 = int(positions.dtype == torch.int64)
        st += ps
    else:
        st += [0, 0]
    return B, T, Hq, Hk, d, rot, st, pos64, _CODE[wt or q.dtype]


def qk_norm_fwd(q, k=None, q_weight=None, k_weight=None, *, kind="l2", eps=1e-6, q_scale=1.0,
                positions=None, inv_freq=None, rotary="half", rotary_scale=1.0, q_out=None,
                k_out=None, stream=None):
    """Norm of every row of q [B, T, H_q, d] and k [B, T, H_k, d] (or None):
    kind "l2" (x / max(|x|, eps)) or "rms" (optional weights [d]); then, with
    inv_freq (float32 [rot / 2], rot <= d), the rotation of the first rot elements by
    positions (int32 or int64 [B, T]; None: 0 .. T-1) in the "half" or
    "interleaved" layout, scaled by rotary_scale; then q_scale on q. Returns
    (q_out, k_out); each may be its dense input. T = 1 is the single-token form."""
    code, dev = _first("q", q, 4)
    B, T, Hq, Hk, d, rot, st, pos64, wcode = _norm_params(q, k, q_weight, k_weight, kind, positions, inv_freq,
                                                          rotary, dev)
    own = (q.dtype,)
    _dense("q_out", q_out, (B, T, Hq, d), own, dev)
    if k_out is not None and k is None:
        raise ValueError("k_out without k")
    _dense("k_out", k_out, (B, T, Hk, d), own, dev)
    if q_out is not None or k_out is not None:
        ins = (("q_weight", q_weight), ("k_weight", k_weight), ("positions", positions), ("inv_freq", inv_freq))
        _apart("q_out", q_out, ins + (("q", q), ("k", k), ("k_out", k_out)), q)
        _apart("k_out", k_out, ins + (("q", q), ("k", k)), k)
    at = _Where(dev, stream)
    if q_out is None:
        q_out = at.empty((B, T, Hq, d), q.dtype)
    if k is not None and k_out is None:
        k_out = at.empty((B, T, Hk, d), q.dtype)
    at.run(_lib.gdr_qk_norm_fwd, q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, _i64(*st), B, T, Hq, Hk,
           d, rot, _NORM[kind], _ROTARY[rotary], eps, q_scale, rotary_scale, pos64, code, wcode)
    return q_out, k_out


def qk_norm_bwd(q, k=None, q_weight=None, k_weight=None, *, dq, dk=None, kind="l2", eps=1e-6,
                q_scale=1.0, positions=None, inv_freq=None, rotary="half", rotary_scale=1.0,
                workspace=None, stream=None):
    """Backward of qk_norm_fwd for the same inputs: dq, dk are the gradients of
    its results, in q's dtype or float32 (both alike). Returns a dict with dq,
    dk, dq_weight and dk_weight (None for what was absent)."""
    code, dev = _first("q", q, 4)
    B, T, Hq, Hk, d, rot, st, pos64, wcode = _norm_params(q, k, q_weight, k_weight, kind, positions, inv_freq,
                                                          rotary, dev)
    st += _check("dq", dq, (B, T, Hq, d), (q.dtype, torch.float32), dev)[:3]
    if (dk is None) != (k is None):
        raise ValueError("dk is given exactly when k is")
    st += (0, 0, 0) if dk is None else _check("dk", dk, (B, T, Hk, d), (dq.dtype,), dev)[:3]
    at, f32 = _Where(dev, stream), torch.float32
    g = {"dq": at.empty((B, T, Hq, d), f32), "dk": None if k is None else at.empty((B, T, Hk, d), f32),
         "dq_weight": None if q_weight is None else at.empty((d,), f32),
         "dk_weight": None if k_weight is None else at.empty((d,), f32)}
    ws, nbytes = None, 0
    if q_weight is not None or k_weight is not None:
        ws, nbytes = at.scratch(workspace, _lib.gdr_qk_norm_bwd_workspace_size(d))
    at.run(_lib.gdr_qk_norm_bwd, q, k, q_weight, k_weight, positions, inv_freq, dq, dk, g["dq"], g["dk"],
           g["dq_weight"], g["dk_weight"], ws, nbytes, _i64(*st), B, T, Hq, Hk, d, rot, _NORM[kind], _ROTARY[rotary],
           eps, q_scale, rotary_scale, pos64, code, wcode, _CODE[dq.dtype])
    return g
