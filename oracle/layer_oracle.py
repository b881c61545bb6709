"""Float64 oracle of the operators around the attention call: rotary positions with
several axes, per-head query/key norms with the rotation, the gradient of that pass,
and the matrix product with bias, activation, gate and residual. Plain numpy, written
from the formulas; shares no code with the GPU path.

Tensors are [B, H, N, d]; a rope is a dict(dims, lens, start, scale, theta, style, first).
"""
from __future__ import annotations

import math

import numpy as np


def rope(dims, lens, theta=10000.0, start=(0, 0, 0), scale=(1, 1, 1), style="interleaved", first=0):
    return dict(dims=dims, lens=lens, theta=theta, start=start, scale=scale, style=style, first=first)


def angles(r, B, N, d, pos=None):
    """[B, N, d/2] angles; tokens outside the grid and pairs no axis owns get 0."""
    out = np.zeros((B, N, d // 2))
    off = 0
    for a, (da, la) in enumerate(zip(r["dims"], r["lens"])):
        inner = int(np.prod(r["lens"][a + 1:], dtype=np.int64))
        for j in range(da // 2):
            f = r["theta"] ** (-2.0 * j / da)
            if pos is None:
                n = np.arange(int(np.prod(r["lens"], dtype=np.int64)))
                p = (n // inner) % la
                out[:, r["first"]:r["first"] + n.size, off + j] = (r["start"][a] + p) * r["scale"][a] * f
            else:
                out[:, :, off + j] = (r["start"][a] + pos[:, :, a]) * r["scale"][a] * f
        off += da // 2
    return out


def _pair_index(r, d):
    R = sum(r["dims"])
    i = np.arange(R // 2)
    if r["style"] == "interleaved":
        return 2 * i, 2 * i + 1
    return i, i + R // 2


def rotate(x, r, pos=None, inverse=False):
    B, H, N, d = x.shape
    ang = angles(r, B, N, d, pos)[:, None]
    if inverse:
        ang = -ang
    ia, ib = _pair_index(r, d)
    c, s = np.cos(ang)[..., :ia.size], np.sin(ang)[..., :ia.size]
    y = x.copy()
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ia] * s + x[..., ib] * c
    return y


def pair_size(x, r):
    """|x0| + |x1| of each element's pair: the scale of a rotation's rounding errors."""
    ia, ib = _pair_index(r, x.shape[-1])
    y = np.abs(x)
    y[..., ia] = y[..., ib] = np.abs(x[..., ia]) + np.abs(x[..., ib])
    return y


def norm_rotate(x, w, eps, r, pos=None):
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotate(x * rstd * w, r, pos)


def norm_rotate_grad(x, w, eps, dy, r, pos=None):
    """(dx, dw) for y = norm_rotate(x, w, eps, r, pos)."""
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * rstd
    g = rotate(dy, r, pos, inverse=True)
    dx = rstd * (g * w - xh * (g * w * xh).mean(-1, keepdims=True))
    return dx, (g * xh).sum((0, 1, 2))


_erfc = np.vectorize(math.erfc, otypes=[float])


def logistic(t):
    return np.where(t >= 0, 1.0 / (1.0 + np.exp(-np.abs(t))), np.exp(-np.abs(t)) / (1.0 + np.exp(-np.abs(t))))


def activate(z, act):
    if act == "gelu_tanh":
        return z * logistic(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "gelu_erf":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    if act == "silu":
        return z * logistic(z)
    return z


def linear(x, w, bias=None, gate=None, residual=None, act="none"):
    """x: [B, N, in] or the attention's [B, heads, N, d]; returns (y, z) with z before the activation."""
    if x.ndim == 4:
        B, h, N, d = x.shape
        x = x.transpose(0, 2, 1, 3).reshape(B, N, h * d)
    z = x @ w.T + (0.0 if bias is None else bias)
    y = activate(z, act)
    if gate is not None:
        y = gate[:, None, :] * y
    if residual is not None:
        y = residual + y
    return y, z
