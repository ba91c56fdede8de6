"""Plain float64 definitions of the operators round the layer: layer norm, gradient clipping, and the
experts' FFN with 4-bit weights.  Shares no code with the library."""
from __future__ import annotations

import math

import numpy as np

__all__ = ["layer_norm", "layer_norm_backward", "grad_norm", "clip_factor", "quantize_w4", "pack_w4", "w4_values",
           "w4_ffn"]

GROUP = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def layer_norm(x, w, b, eps):
    """(y, mean, rstd) of rows x [rows, H]; w, b [H] or None."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if b is not None:
        y = y + np.asarray(b, np.float64)
    return y, mean, rstd


def layer_norm_backward(dy, x, w, mean, rstd):
    """(dx, dw, db) with the statistics given."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    n = (x - np.asarray(mean, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    g = dy if w is None else dy * np.asarray(w, np.float64)
    dx = np.asarray(rstd, np.float64)[:, None] * (
        g - g.mean(1, keepdims=True) - n * (g * n).mean(1, keepdims=True))
    return dx, (dy * n).sum(0), dy.sum(0)


def grad_norm(grads):
    return math.sqrt(math.fsum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads))


def clip_factor(norm, max_norm):
    return 1.0 if norm <= max_norm else max_norm / norm


def quantize_w4(w):
    """w [Kin, N] float -> codes [Kin, N], scales [Kin/32, N] (uint8).  Nearest of the eight
    magnitudes by distance, halfway to the even code; 255 for a group that is not finite."""
    w = np.asarray(w, np.float64)
    Kin, N = w.shape
    v = w.reshape(Kin // GROUP, GROUP, N)
    fine = np.isfinite(v).all(1, keepdims=True)
    v = np.where(fine, v, 0.0)
    top = np.abs(v).max(1, keepdims=True)
    e = np.where(top > 0, np.maximum(np.frexp(top)[1] - 1 - 2, -126), -126)
    d = np.abs(np.ldexp(np.abs(v), -e)[..., None] - E2M1)
    near = d == d.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    c = np.where(near.sum(-1) > 1, even.argmax(-1), near.argmax(-1)) | np.where(np.signbit(v), 8, 0)
    codes = np.where(fine, c, 0).astype(np.uint8).reshape(Kin, N)
    scales = np.where(fine, e + 127, 255).astype(np.uint8).reshape(Kin // GROUP, N)
    return codes, scales


def pack_w4(codes, scales):
    """The layout of the C header: (code bytes, scale bytes) of one matrix, flat."""
    Kin, N = codes.shape
    kb, sb = -(-Kin // 128), -(-Kin // 512)
    cb = np.zeros((N // 16, kb, 4, 16, 16), np.uint8)
    sc = np.full((N // 16, sb, 4, 16, 4), 127, np.uint8)
    for k in range(Kin):
        for n in range(N):
            cb[n // 16, k // 128, k % 128 // 32, n % 16, k % 32 // 2] |= int(codes[k, n]) << (4 * (k % 2))
    for g in range(Kin // GROUP):
        for n in range(N):
            sc[n // 16, g // 16, g % 4, n % 16, g // 4 % 4] = scales[g, n]
    return cb.reshape(-1), sc.reshape(-1)


def w4_values(codes, scales):
    """[Kin, N] float64 that codes and scales stand for."""
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, GROUP, axis=0)


def w4_ffn(x, topk, gates, w13, w2):
    """out [T, H] and a bound of what float32 sums and the two-term activation may be off, elementwise
    (without the rounding of the output).  w13 [E, H, 2I], w2 [E, I, H] float64."""
    x, gates = np.asarray(x, np.float64), np.asarray(gates, np.float64)
    T, H = x.shape
    E, _, I2 = w13.shape
    I, u = I2 // 2, 2.0 ** -24
    out, off, mass = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for k, e in enumerate(topk[t]):
            if not 0 <= e < E:
                continue
            gu = x[t] @ w13[e]
            # a sum of H products in any order, each step rounded to float32
            dgu = H * u * (np.abs(x[t]) @ np.abs(w13[e]))
            g, v = gu[:I], gu[I:]
            s = g / (1 + np.exp(-g))
            a = s * v
            # |silu'| < 1.1; exponential, sum, quotient and product within 8 roundings; two bf16 terms 2^-15
            da = 1.1 * dgu[:I] * (np.abs(v) + dgu[I:]) + np.abs(s) * dgu[I:] + np.abs(a) * (8 * u + 2.0 ** -15)
            y = a @ w2[e]
            dy = da @ np.abs(w2[e]) + (2 * I + 1) * u * ((np.abs(a) + da) @ np.abs(w2[e]))
            out[t] += gates[t, k] * y
            off[t] += np.abs(gates[t, k]) * dy
            mass[t] += np.abs(gates[t, k]) * (np.abs(y) + dy)
    return out, off + (len(topk[0]) + 1) * u * mass
