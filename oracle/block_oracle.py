"""Block operators in numpy, 64 bits: layer norm, the linear layer and its
gradients, and the 8-bit activation checkpoint format.  Written from the
formulas in ``include/fsdp_unit.h``; shares no code with the library."""
from __future__ import annotations

import math

import numpy as np

GROUP = 32


# ---- 8-bit checkpoints -------------------------------------------------------

def act8_pack(x):
    """(q int8 [rows, 32*ceil(cols/32)], byte uint8 [rows, ceil(cols/32)])."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    q = np.zeros((rows, groups * GROUP), np.int8)
    byte = np.zeros((rows, groups), np.uint8)
    for r in range(rows):
        for g in range(groups):
            v = x[r, g * GROUP:(g + 1) * GROUP]
            if not np.all(np.isfinite(v)):
                byte[r, g] = 255
                continue
            a = float(np.max(np.abs(v)))
            E = -120 if a == 0 else max(-120, min(127, math.frexp(a)[1] - 1))
            byte[r, g] = E + 127
            q[r, g * GROUP:g * GROUP + v.size] = np.clip(np.rint(np.ldexp(v, 6 - E)), -127, 127)
    return q, byte


def act8_unpack(q, byte, cols):
    e = byte.astype(np.int32) - 133
    v = np.ldexp(q.astype(np.float64).reshape(byte.shape + (GROUP,)), e[..., None])
    v[byte == 255] = np.nan
    return v.reshape(q.shape)[:, :cols]


# ---- activations --------------------------------------------------------------

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "none":
        return z
    if kind == "relu":
        return np.where(np.isnan(z), np.nan, np.maximum(z, 0.0))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))


def slope(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "none":
        return np.ones_like(z)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = np.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)
    return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)


# ---- layer norm ---------------------------------------------------------------

def layer_norm(x, gamma, beta, eps):
    x = np.asarray(x, np.float64)
    mean = x.sum(axis=1) / x.shape[1]
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).sum(axis=1) / x.shape[1] + eps)
    return d * rstd[:, None] * gamma + beta, mean, rstd


def layer_norm_grad(dy, x, gamma, mean, rstd, add=None):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    dx = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - xh * (g * xh).mean(axis=1, keepdims=True))
    if add is not None:
        dx = dx + add
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


# ---- linear layer (w is in_features x out_features) ---------------------------

def linear(x, w, bias=None, kind="none", residual=None):
    """(y, z)."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64)
    if bias is not None:
        z = z + bias
    y = activation(z, kind)
    return (y if residual is None else y + residual), z


def linear_grad_input(dy, w, kind="none", z=None, add=None):
    dx = np.asarray(dy, np.float64) @ np.asarray(w, np.float64).T
    if kind != "none":
        dx = dx * slope(z, kind)
    return dx if add is None else dx + add


def linear_grad_weight(x, dy):
    """(dw, dbias)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    return x.T @ dy, dy.sum(axis=0)
