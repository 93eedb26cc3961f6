"""Plain NumPy oracle of the operators around the experts, in 64 bits: the
norm with its quantized outputs, the balance loss, the gradients of the
router, the combine and the norm, and the Newton-Schulz iteration.

Written from the definitions; shares nothing with the HIP library.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
# the values of E4M3 from 0 up (OCP, no infinities): subnormal steps of 2^-9, then 8 per octave up to 448
E4M3 = np.array([m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8) if (e, m) != (8, 7)])


def rms_norm(s, weight, eps):
    """-> (y, r) of the rows of s."""
    s = np.asarray(s, np.float64)
    r = 1 / np.sqrt((s * s).mean(-1) + eps)
    return s * r[..., None] * np.asarray(weight, np.float64), r


def rms_norm_grad(dy, s, weight, eps, dsum=0.0):
    """-> (dx, dweight)."""
    dy, s, weight = (np.asarray(a, np.float64) for a in (dy, s, weight))
    r = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    d, n = dy * weight, s * r
    return r * (d - n * (d * n).mean(-1, keepdims=True)) + dsum, (dy * n).sum(0)


def mxfp8_bytes(amax):
    """E8M0 bytes of MXFP8 blocks with largest magnitudes `amax` (NaN or inf -> 255)."""
    amax = np.asarray(amax, np.float64)
    bad = ~np.isfinite(amax)
    _, e = np.frexp(np.where(bad, 1.0, amax))
    e = np.where(np.where(bad, 1.0, amax) > 0, np.maximum(e - 1 - 8, -127), -127)
    return np.where(bad, 255, e + 127).astype(np.uint8)


def round_e4m3(v):
    """Magnitude code (0..126) of the E4M3 value nearest to v >= 0, ties to the even code, saturating."""
    v = np.minimum(np.asarray(v, np.float64), E4M3[-1])
    hi = np.clip(np.searchsorted(E4M3, v), 1, len(E4M3) - 1)
    up, down = E4M3[hi] - v, v - E4M3[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantize_mxfp8(x, scales=None):
    """x [..., cols] -> (codes uint8 [..., cols], scale bytes [..., cols/32])."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    with np.errstate(invalid="ignore"):
        amax = np.where(np.isnan(b).any(-1), np.nan, np.abs(b).max(-1))
    s = mxfp8_bytes(amax) if scales is None else scales
    bad = (s == 255)[..., None]
    unit = np.exp2(np.where(s == 255, 0.0, s.astype(np.float64) - 127))[..., None]
    code = round_e4m3(np.where(bad, 0.0, np.abs(np.nan_to_num(b)) / unit)) | (np.signbit(b).astype(np.int64) << 7)
    return np.where(bad, 0, code).reshape(x.shape).astype(np.uint8), s


def dequantize_mxfp8(codes, scales):
    v = np.append(E4M3, np.nan)[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    unit = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v.reshape(*scales.shape, BLOCK) * unit[..., None]).reshape(codes.shape)


def softmax(logits):
    """Over the last axis; a row of -inf alone gives zeros."""
    l = np.asarray(logits, np.float64)
    m = l.max(-1, keepdims=True)
    e = np.exp(l - np.where(np.isneginf(m), 0.0, m))
    s = e.sum(-1, keepdims=True)
    return e / np.where(s == 0, 1.0, s)


def expert_counts(ids, E, mask):
    kept = ids[mask].reshape(-1)
    return np.bincount(kept[(kept >= 0) & (kept < E)], minlength=E)


def balance_loss(logits, ids, coef, mask=None):
    """-> (loss, counts, slope)."""
    T, E = logits.shape
    mask = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    n, counts = int(mask.sum()), expert_counts(ids, E, mask)
    slope = coef * E * counts / (ids.shape[1] * max(n, 1) ** 2)
    return float((slope * softmax(logits[mask]).sum(0)).sum()), counts, slope


def route_grad(logits, ids, dw=None, slope=None, dloss=1.0, mask=None):
    """Gradient of the logits."""
    T, E = logits.shape
    mask = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    dp = np.zeros((T, E))
    if slope is not None:
        dp += dloss * np.asarray(slope, np.float64)
    if dw is not None:
        for j in range(ids.shape[1]):
            ok = (ids[:, j] >= 0) & (ids[:, j] < E)
            np.add.at(dp, (np.nonzero(ok)[0], ids[ok, j]), np.asarray(dw, np.float64)[ok, j])
    p = softmax(logits)
    return np.where(mask[:, None], p * (dp - (p * dp).sum(-1, keepdims=True)), 0.0)


def newton_schulz(g, steps, coefficients, eps):
    """X <- a X + (b A + c A^2) X with A = X X^T from X = g / (|g| + eps), for each matrix."""
    a, b, c = coefficients
    x = np.asarray(g, np.float64)
    x = x / (np.sqrt((x * x).sum((-2, -1), keepdims=True)) + eps)
    for _ in range(steps):
        s = x @ np.swapaxes(x, -1, -2)
        x = a * x + (b * s + c * s @ s) @ x
    return x
