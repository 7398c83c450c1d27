"""The norms around a block in float64 (qlora_block_norm_fwd / _bwd).

Per token row, o = w_offset:
  nh = h rstd_post, rstd_post = (mean h^2 + eps)^-1/2    (nh = h without w_post)
  x' = alpha x + gate[m // gate_rows] (o + w_post) nh
  y  = x' rstd_pre (o + w_pre), rstd_pre = (mean x'^2 + eps)^-1/2
The device rounds x' to its type before the norm reads it, so `pre` takes the
stored x'.  The backward is the chain rule written out; tests/ checks it
against central differences.
"""
from __future__ import annotations

import numpy as np


def _gate(gate, gate_rows, M):
    return None if gate is None else gate[np.arange(M) // gate_rows]


def post(x, h, w_post=None, gate=None, gate_rows=0, alpha=1.0, eps=1e-6, w_offset=0.0):
    """x' (unrounded) and rstd_post (None without w_post)."""
    rstd, branch = None, h
    if w_post is not None:
        rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
        branch = h * rstd[:, None] * (w_offset + w_post)
    if gate is not None:
        branch = branch * _gate(gate, gate_rows, h.shape[0])
    return alpha * x + branch, rstd


def pre(x_out, w_pre, eps=1e-6, w_offset=0.0):
    """y (unrounded) and rstd_pre from the stored x'."""
    rstd = 1.0 / np.sqrt(np.mean(x_out * x_out, axis=1) + eps)
    return x_out * rstd[:, None] * (w_offset + w_pre), rstd


def backward(x_out, h, dx_out, dy, w_pre=None, w_post=None, gate=None, gate_rows=0, alpha=1.0, eps=1e-6, w_offset=0.0):
    """Gradients of <dx_out, x'> + <dy, y>; dy or dx_out may be None (zero).
    Also the sums of absolute values that bound the error of an fp32 evaluation
    (keys ending in _abs)."""
    M, D = (dy if dy is not None else dx_out).shape
    dr = np.zeros((M, D)) if dx_out is None else dx_out.copy()
    dr_abs = np.abs(dr)
    out = {}
    n = np.zeros((M, D))
    if dy is not None:
        rstd = 1.0 / np.sqrt(np.mean(x_out * x_out, axis=1, keepdims=True) + eps)
        n = x_out * rstd
        out["dw_pre"] = np.sum(dy * n, axis=0)
        out["dw_pre_abs"] = np.sum(np.abs(dy * n), axis=0)
        dn = dy * (w_offset + w_pre)
        dr = dr + rstd * (dn - n * np.mean(dn * n, axis=1, keepdims=True))
        dr_abs = dr_abs + rstd * (np.abs(dn) + np.abs(n) * np.mean(np.abs(dn * n), axis=1, keepdims=True))
    out["dx"], out["dx_abs"] = alpha * dr, abs(alpha) * dr_abs
    if h is None:
        if gate is not None:
            dr, dr_abs = dr * _gate(gate, gate_rows, M), dr_abs * np.abs(_gate(gate, gate_rows, M))
        if w_post is None:
            out["dh"], out["dh_abs"] = dr, dr_abs
        return out
    rstd = None if w_post is None else 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    nh = h if rstd is None else h * rstd
    w = 1.0 if w_post is None else w_offset + w_post
    g = _gate(gate, gate_rows, M) if gate is not None else np.ones((1, 1))
    S, S_abs = dr * nh, dr_abs * np.abs(nh)
    if gate is not None:
        index = np.arange(M) // gate_rows
        out["dgate"] = np.zeros(gate.shape)
        out["dgate_abs"] = np.zeros(gate.shape)
        np.add.at(out["dgate"], index, S * w)
        np.add.at(out["dgate_abs"], index, S_abs * np.abs(w))
    dnh, dnh_abs = dr * g * w, dr_abs * np.abs(g * w)
    if w_post is None:
        out["dh"], out["dh_abs"] = dnh, dnh_abs
        return out
    out["dw_post"] = np.sum(S * g, axis=0)
    out["dw_post_abs"] = np.sum(S_abs * np.abs(g), axis=0)
    out["dh"] = rstd * (dnh - nh * np.mean(dnh * nh, axis=1, keepdims=True))
    out["dh_abs"] = rstd * (dnh_abs + np.abs(nh) * np.mean(dnh_abs * np.abs(nh), axis=1, keepdims=True))
    return out
