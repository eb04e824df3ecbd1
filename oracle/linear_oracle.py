"""Float64 numpy statement of the linear map with bias, activation and residual,
of its gradients, and of the 8-bit activation checkpoint (include/prism.h).
Used by the tests only; shares no code with the library."""
from __future__ import annotations

import numpy as np

NONE, RELU, SILU, GELU = 0, 1, 2, 3
_K = np.sqrt(2.0 / np.pi)


def _logistic(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def act(z, kind):
    if kind == RELU:
        return np.maximum(z, 0.0)
    if kind == SILU:
        return z * _logistic(z)
    if kind == GELU:
        return 0.5 * z * (1.0 + np.tanh(_K * (z + 0.044715 * z ** 3)))
    return z


def slope(z, kind):
    """d act / dz."""
    if kind == RELU:
        return (z > 0).astype(np.float64)
    if kind == SILU:
        p = _logistic(z)
        return p + z * p * (1.0 - p)
    if kind == GELU:
        t = np.tanh(_K * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _K * (1.0 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def forward(X, W, bias=None, kind=NONE, R=None):
    """(Z, Y)."""
    Z = X @ W.T
    if bias is not None:
        Z = Z + bias
    Y = act(Z, kind)
    return Z, (Y if R is None else Y + R)


def backward(dY, X, W, Z, kind):
    """(dZ, dX, dW, db)."""
    dZ = dY if kind == NONE else dY * slope(Z, kind)
    return dZ, dZ @ W, dZ.T @ X, dZ.sum(axis=0)


def ckpt8_pack(x):
    """x [n, width] -> (codes int8 [n, ld], scale bytes uint8 [n, ld / 32])
    with ld = width rounded up to 128; channels past width count as 0."""
    n, width = x.shape
    ld = (width + 127) // 128 * 128
    b = np.zeros((n, ld), np.float64)
    b[:, :width] = x
    b = b.reshape(n, ld // 32, 32)
    codes = np.zeros(b.shape, np.int8)
    scales = np.zeros(b.shape[:2], np.uint8)
    for idx in np.ndindex(*b.shape[:2]):
        v = b[idx]
        if not np.isfinite(v).all():
            scales[idx] = 255
            continue
        s = 1
        top = np.abs(v).max()
        if top > 0:
            s = max(1, int(np.floor(np.log2(top / 127.0))) + 127)
            while top > 127.0 * 2.0 ** (s - 127):
                s += 1
            while s > 1 and top <= 127.0 * 2.0 ** (s - 128):
                s -= 1
        s = min(s, 248)
        scales[idx] = s
        codes[idx] = np.rint(np.clip(v * 2.0 ** (127 - s), -127, 127)).astype(np.int8)
    return codes.reshape(n, ld), scales


def ckpt8_unpack(codes, scales, width):
    with np.errstate(invalid="ignore"):
        q = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (codes.reshape(codes.shape[0], -1, 32) * q[..., None]).reshape(codes.shape[0], -1)[:, :width]
