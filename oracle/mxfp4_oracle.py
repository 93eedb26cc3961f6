"""Plain NumPy oracle of the MXFP4 codec, the grouped MXFP4 product and the
gated expert block with its gradient, in 64 bits.

Written from the definitions (OCP Microscaling: blocks of 32, E8M0 scale,
E2M1 elements); shares nothing with the HIP library.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def block_bytes(amax, rule="floor"):
    """E8M0 bytes of blocks with largest magnitudes `amax` (float64; NaN or inf -> 255)."""
    amax = np.asarray(amax, np.float64)
    bad = ~np.isfinite(amax)
    m, e = np.frexp(np.where(bad, 1.0, amax))  # amax = m 2^e with m in [0.5, 1)
    e = e - 1 + ((m >= 0.875) if rule == "even" else 0)  # floor(log2), or that of the rounded magnitude
    e = np.where(np.where(bad, 1.0, amax) > 0, np.clip(e - 2, -127, 125), -127)
    return np.where(bad, 255, e + 127).astype(np.uint8)


def round_e2m1(v):
    """Magnitude index (0..7) of the level nearest to v >= 0, ties to the even index, saturating."""
    v = np.asarray(v, np.float64)
    mid = (LEVELS[1:] + LEVELS[:-1]) / 2
    idx = np.zeros(v.shape, np.int64)
    for i, t in enumerate(mid):  # level i + 1 is taken above the midpoint, and at it when i + 1 is even
        idx += (v >= t) if (i + 1) % 2 == 0 else (v > t)
    return idx


def quantize(x, rule="floor", scales=None):
    """x [..., cols] -> (unpacked codes uint8 [..., cols], scale bytes [..., cols/32])."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    with np.errstate(invalid="ignore"):
        amax = np.where(np.isnan(b).any(-1), np.nan, np.abs(b).max(-1))
    s = block_bytes(amax, rule) if scales is None else scales
    unit = np.exp2(s.astype(np.float64) - 127)[..., None]
    with np.errstate(invalid="ignore"):
        code = round_e2m1(np.abs(b) / unit) | (np.signbit(b).astype(np.int64) << 3)
    code = np.where((s == 255)[..., None], 0, code)
    return code.reshape(x.shape).astype(np.uint8), s


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty((*packed.shape[:-1], packed.shape[-1] * 2), np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def dequantize(codes, scales):
    """Unpacked codes and scale bytes -> float64 values."""
    v = LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    unit = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v.reshape(*scales.shape, BLOCK) * unit[..., None]).reshape(codes.shape)


def grouped(x, w, offsets, row_token=None, magnitude=False):
    """Rows x[t(i)] times w[e(i)]^T (float64); with magnitude=True the sums of |products|."""
    R = len(row_token) if row_token is not None else x.shape[0]
    y = np.zeros((R, w.shape[1]))
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a < b:
            xe = x[row_token[a:b]] if row_token is not None else x[a:b]
            y[a:b] = (np.abs(xe) @ np.abs(w[e]).T) if magnitude else xe @ w[e].T
    return y


def sigmoid(z):
    """1 / (1 + e^-z), as e^z / (1 + e^z) below 0: no cancellation, no overflow."""
    z = np.asarray(z, np.float64)
    e = np.exp(-np.abs(z))
    return np.where(z < 0, e, 1.0) / (1 + e)


def silu(z):
    return z * sigmoid(z)


def gated(gu):
    """h of [gate | up]."""
    g, u = np.split(gu, 2, axis=-1)
    return silu(g) * u


def gated_grad(dh, gu):
    """Gradient of [gate | up] from that of h = silu(gate) * up."""
    g, u = np.split(gu, 2, axis=-1)
    s = sigmoid(g)
    return np.concatenate((dh * u * s * (1 + g * (1 - s)), dh * g * s), axis=-1)
