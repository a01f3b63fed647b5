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

import torch  # noqa: F401  (its libraries, before the module that links to them)

from . import _lib

_lib.load()  # builds what is missing
from . import _layers  # noqa: E402

_layers.set_error(_lib.GdrError)


# ---------------------------------------------------------------- convolution

def conv_fwd(x, weight, bias=None, X0=None, *, activation="silu", lengths=None, out=None,
             final_state=True, X_T=None, stream=None):
    """Short causal depthwise convolution over [B, T, D] inputs: weight [D, W],
    bias [D] (x's dtype or float32), X0 [B, W-1, D] the inputs before the first
    token (None: zeros), activation "silu" or None. Returns (y, X_T), X_T the
    last W - 1 inputs (None when final_state is False); X_T may be X0."""
    return _layers.conv_fwd(x, weight, bias, X0, activation, lengths, out, final_state, X_T, stream)


def conv_bwd(x, weight, bias=None, X0=None, *, dy, dX_T=None, activation="silu", lengths=None,
             workspace=None, need_dX0=True, stream=None):
    """Backward of conv_fwd for the same inputs: dy [B, T, D] in x's dtype or
    float32, dX_T [B, W-1, D] float32 or None. Returns a dict with dx, dweight,
    dbias (None without bias) and dX0 (None without X0 or need_dX0)."""
    return _layers.conv_bwd(x, weight, bias, X0, dy, dX_T, activation, lengths, workspace, need_dX0, stream)


def conv_step(x, weight, bias, X, *, activation="silu", out=None, stream=None):
    """One token per sequence: x [B, D], X [B, W-1, D] the last inputs, moved on
    in place. Returns y [B, D]."""
    return _layers.conv_step(x, weight, bias, X, activation, out, stream)


# ---------------------------------------------------------------- selective scan

def scan_fwd(u, delta, A, Bm, Cm, D=None, z=None, h0=None, *, delta_bias=None, delta_softplus=False,
             lengths=None, workspace="auto", out=None, final_state=True, h_T=None, stream=None):
    """Selective scan over [B, T, D] inputs u and step sizes delta (delta_bias
    [D] added, then softplus with delta_softplus): A [D, N] and D [D] float32,
    Bm, Cm [B, T, G, N] shared by the D / G channels of a group, z [B, T, D] a
    gate (y z sigmoid(z)), h0 [B, D, N] float32 (None: zeros). Returns (y, h_T),
    h_T None when final_state is False; h_T may be h0. workspace: "auto" takes
    from torch what a split of the tokens needs (few channels, many tokens), a
    device tensor supplies it, None leaves the tokens unsplit."""
    return _layers.scan_fwd(u, delta, A, Bm, Cm, D, z, h0, delta_bias, delta_softplus, lengths, workspace, out,
                            final_state, h_T, stream)


def scan_bwd(u, delta, A, Bm, Cm, D=None, z=None, h0=None, *, dy, dh_T=None, delta_bias=None,
             delta_softplus=False, lengths=None, workspace=None, need_dh0=True, stream=None):
    """Backward of scan_fwd for the same inputs: dy [B, T, D] in u's dtype or
    float32, dh_T [B, D, N] float32 or None. Returns a dict with du, ddelta, dA,
    dB, dC, dD, dz, ddelta_bias and dh0 (None for what was absent, dh0 also
    without need_dh0)."""
    return _layers.scan_bwd(u, delta, A, Bm, Cm, D, z, h0, dy, dh_T, delta_bias, delta_softplus, lengths, workspace,
                            need_dh0, stream)


def scan_step(u, delta, A, Bm, Cm, D, z, h, *, delta_bias=None, delta_softplus=False, out=None,
              stream=None):
    """One token per sequence: u, delta, z [B, D], Bm, Cm [B, G, N], h [B, D, N]
    float32 updated in place. Returns y [B, D]."""
    return _layers.scan_step(u, delta, A, Bm, Cm, D, z, h, delta_bias, delta_softplus, out, stream)


# ---------------------------------------------------------------- norm and rotation

def qk_norm_fwd(q, k=None, q_weight=None, k_weight=None, *, kind="l2", eps=1e-6, q_scale=1.0,
                positions=None, inv_freq=None, rotary="half", rotary_scale=1.0, q_out=None,
                k_out=None, stream=None):
    """Norm of every row of q [B, T, H_q, d] and k [B, T, H_k, d] (or None):
    kind "l2" (x / max(|x|, eps)) or "rms" (optional weights [d]); then, with
    inv_freq (float32 [rot / 2], rot <= d), the rotation of the first rot elements by
    positions (int32 or int64 [B, T]; None: 0 .. T-1) in the "half" or
    "interleaved" layout, scaled by rotary_scale; then q_scale on q. Returns
    (q_out, k_out); each may be its dense input. T = 1 is the single-token form."""
    return _layers.qk_norm_fwd(q, k, q_weight, k_weight, kind, eps, q_scale, positions, inv_freq, rotary,
                               rotary_scale, q_out, k_out, stream)


def qk_norm_bwd(q, k=None, q_weight=None, k_weight=None, *, dq, dk=None, kind="l2", eps=1e-6,
                q_scale=1.0, positions=None, inv_freq=None, rotary="half", rotary_scale=1.0,
                workspace=None, stream=None):
    """Backward of qk_norm_fwd for the same inputs: dq, dk are the gradients of
    its results, in q's dtype or float32 (both alike). Returns a dict with dq,
    dk, dq_weight and dk_weight (None for what was absent)."""
    return _layers.qk_norm_bwd(q, k, q_weight, k_weight, kind, eps, q_scale, positions, inv_freq, rotary,
                               rotary_scale, dq, dk, workspace, stream)
