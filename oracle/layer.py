"""fp64 reference of the layer around the recurrence: projections with their epilogue, the norms
around a block, the output norm with its gate, and their gradients.

TEST INFRASTRUCTURE ONLY, like the rest of `oracle/`: it shares no code with the CUDA library.
The gradients are written from the formulas of rms(a) = a / sqrt(mean(a^2) + eps); the tests
compare them with differences of the forward.
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def _sigmoid(z):
    return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))


def act(kind, z):
    z = np.asarray(z, np.float64)
    return {"none": lambda: z, "relu": lambda: np.maximum(z, 0), "silu": lambda: z * _sigmoid(z),
            "gelu": lambda: z * 0.5 * (1 + _erf(z / math.sqrt(2))),
            "sigmoid": lambda: _sigmoid(z)}[kind]()


def act_grad(kind, z):
    z = np.asarray(z, np.float64)
    p = _sigmoid(z)
    return {"none": lambda: np.ones_like(z), "relu": lambda: (z > 0).astype(np.float64),
            "silu": lambda: p + z * p * (1 - p), "sigmoid": lambda: p * (1 - p),
            "gelu": lambda: 0.5 * (1 + _erf(z / math.sqrt(2)))
            + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)}[kind]()


def linear(x, w, bias=None, activation="none", residual=None, scale=1.0):
    """Returns (y, z)."""
    z = x @ w.T + (0 if bias is None else bias)
    return scale * act(activation, z) + (0 if residual is None else residual), z


def linear_bwd(x, w, d_y, z=None, activation="none", scale=1.0):
    """Returns (dx, dw, dbias, dz)."""
    dz = scale * d_y * (1 if activation == "none" else act_grad(activation, z))
    return dz @ w, dz.T @ x, dz.sum(0), dz


def rms(a, eps):
    r = 1 / np.sqrt(np.mean(a * a, -1, keepdims=True) + eps)
    return a * r, r


def _rms_vjp(a, eps, d):
    n, r = rms(a, eps)
    return r * (d - n * np.mean(d * n, -1, keepdims=True))


def residual_norm(x, weight=None, residual=None, post_weight=None, gate=None, scale=1.0, eps=1e-6):
    """Returns (y or None, h)."""
    u = x if post_weight is None else rms(x, eps)[0] * post_weight
    h = scale * u * (1 if gate is None else gate) + (0 if residual is None else residual)
    return (None if weight is None else rms(h, eps)[0] * weight), h


def residual_norm_bwd(x, h, weight, d_y, d_h=None, post_weight=None, gate=None, scale=1.0, eps=1e-6):
    """Returns (dx, d_residual, d_weight, d_post_weight, d_gate), d_gate per element (the caller
    sums it over tokens for a [N] gate)."""
    dh = np.zeros_like(h) if d_h is None else d_h.copy()
    dw = None
    if weight is not None:
        dw = (d_y * rms(h, eps)[0]).sum(0)
        dh = dh + _rms_vjp(h, eps, d_y * weight)
    u = x if post_weight is None else rms(x, eps)[0] * post_weight
    du = scale * dh * (1 if gate is None else gate)
    dg = None if gate is None else scale * dh * u
    if post_weight is None:
        return du, dh, dw, None, dg
    return _rms_vjp(x, eps, du * post_weight), dh, dw, (du * rms(x, eps)[0]).sum(0), dg


def gated_norm(o, gate, weight, activation="sigmoid", eps=1e-6):
    return rms(o, eps)[0] * weight * act(activation, gate)


def gated_norm_bwd(o, gate, weight, d_y, activation="sigmoid", eps=1e-6):
    """Returns (d_o, d_gate, d_weight)."""
    n = rms(o, eps)[0]
    dn = d_y * act(activation, gate)
    return (_rms_vjp(o, eps, dn * weight), d_y * n * weight * act_grad(activation, gate),
            (dn * n).reshape(-1, o.shape[-1]).sum(0))
