"""The linear-layer operators written out in float64 (numpy): the definition
the GPU kernels are compared with.

Nothing here is shared with the CUDA path. Inputs are float64 arrays holding the
exact values of the 16- or 8-bit operands; results are not rounded, except by
:func:`quantise_e4m3`, which rounds to the 8-bit grid. Every gradient is the
derivative of the forward function beside it (the tests check that by central
differences).
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def to64(t) -> np.ndarray:
    """Exact float64 values of a torch tensor (16-bit, float8 or float32)."""
    import torch
    if t.dtype is torch.float8_e4m3fn:
        return decode_e4m3(t.detach().cpu().contiguous().view(torch.uint8).numpy())
    return t.detach().cpu().to(torch.float64).numpy()


def _logistic(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def act(z, name):
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * _logistic(z)
    return z


def act_slope(z, name):
    if name == "relu":
        return np.where(np.isnan(z), z, (z > 0).astype(np.float64))
    if name == "gelu":
        return (0.5 * _erfc(-z / math.sqrt(2.0))
                + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = _logistic(z)
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def linear(A, B, alpha=1.0, bias=None, act_name=None, residual=None, scale_a=None, scale_b=None):
    """(D, Z) of D = act(Z) + residual, Z = alpha * scales * A B + bias (A: M x K,
    B: K x N)."""
    z = alpha * (A @ B)
    if scale_a is not None:
        z = z * scale_a[:, None]
    if scale_b is not None:
        z = z * scale_b[None, :]
    if bias is not None:
        z = z + bias[None, :]
    d = act(z, act_name)
    return (d if residual is None else d + residual), z


def linear_grad(dD, Z, act_name=None):
    """(dZ, dbias) from the gradient dD of act(Z)."""
    dz = dD * act_slope(Z, act_name) if act_name not in (None, "none") else dD
    return dz, dz.sum(axis=0)


def rms_norm(X, W=None, residual=None, eps=0.0):
    """(Y, H, rstd)."""
    h = X if residual is None else X + residual
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    y = h * rstd[:, None]
    return (y if W is None else y * W[None, :]), h, rstd


def rms_norm_grad(dY, H, rstd, W=None, dH=None):
    """(dX, dW)."""
    n = H * rstd[:, None]
    g = dY if W is None else dY * W[None, :]
    dx = rstd[:, None] * (g - n * (g * n).mean(axis=1, keepdims=True))
    return (dx if dH is None else dx + dH), (dY * n).sum(axis=0)


def round_e4m3(x):
    """x rounded to the e4m3 grid, ties to even, saturating at 448."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.abs(x)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.where(mag > 0, mag, 1.0)))
    step = np.exp2(np.maximum(e, -6.0) - 3.0)
    return np.clip(np.rint(x / step) * step, -E4M3_MAX, E4M3_MAX)


def quantise_e4m3(y, least=1e-30):
    """(q, scale) per row: scale = max |y| / 448, q = round_e4m3(y / scale); rows
    below `least` get scale 0 and zeros."""
    top = np.abs(y).max(axis=1)
    scale = np.where(top < least, 0.0, top / E4M3_MAX)
    safe = np.where(scale == 0.0, 1.0, scale)
    q = round_e4m3(y / safe[:, None])
    return np.where(scale[:, None] == 0.0, 0.0, q), scale


def decode_e4m3(bits) -> np.ndarray:
    """Values of e4m3 bytes: sign, 4 exponent bits (bias 7), 3 fraction bits;
    exponent 0 is subnormal, 0x7f / 0xff are NaN."""
    b = np.asarray(bits, dtype=np.int64)
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * np.exp2(e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)
