"""Plain float64 definitions of routing, sorting by expert, the weighted combine's gradient, and the
experts' FFN with 8-bit weights.  Shares no code with the library.

Where a function also returns a bound, it is how far an evaluation in float32 may be off: u = 2^-24 is half
a step of float32, and a bound names the roundings that it counts."""
from __future__ import annotations

import numpy as np

__all__ = ["route", "route_backward", "sort_pairs", "combine_backward", "e4m3", "quantize_fp8", "pack_fp8", "fp8_values",
           "round_rows", "fp8_ffn"]

U = 2.0 ** -24
BLOCK = 128


# -- routing -----------------------------------------------------------------

def _shares(z, ids, mode):
    """(p [K], rel [K]): shares of the picks of one row, and their relative error in float32 over u.

    An exponential of a difference d is off by |d| (the difference's own rounding) and 2 more; a sum by the weighted
    mean of its terms' errors and its longest chain; a quotient by one."""
    on = ids >= 0
    at = np.where(on, ids, 0)
    w = np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z))) if mode == "sigmoid" else z
    # a log-sigmoid is two functions of 2 roundings each and a sum: off by 4 of its size and of log 2
    extra = 4 * (np.abs(w) + 1) if mode == "sigmoid" else np.zeros_like(w)
    picked = np.where(on, w[at], -np.inf)
    base, be = (w, extra) if mode == "softmax_all" else (picked, np.where(on, extra[at], 0))
    fin = base > -np.inf
    if not on.any() or not fin.any():
        return np.zeros(len(ids)), np.zeros(len(ids))
    top = base.max()
    t = np.exp(np.where(fin, base - top, -np.inf))
    d = np.where(fin, top - np.where(fin, base, 0), 0) + 2 + be + be[base.argmax()]
    S = t.sum()
    chain = len(base) / 16 + 8
    p = np.where(on, np.exp(picked - top) / S, 0.0)
    real = on & (picked > -np.inf)           # a share of exactly 0 is off by nothing
    own = np.where(real, top - np.where(real, picked, 0), 0) + 2 + np.where(on, extra[at], 0) + be[base.argmax()]
    return p, own + (t * d).sum() / S + chain + 2


def route(logits, bias, K, mode, scale=1.0):
    """(ids [T, K], gates, bound of the gates) of logits [T, E], finite or -inf."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    ids, gates, tol = np.full((T, K), -1, np.int32), np.zeros((T, K)), np.zeros((T, K))
    for t in range(T):
        key = z[t].copy()
        if bias is not None:
            with np.errstate(over="ignore"):
                key = (1 / (1 + np.exp(-z[t])) if mode == "sigmoid" else z[t]) + np.asarray(bias, np.float64)
            key[z[t] == -np.inf] = -np.inf
        order = sorted((e for e in range(E) if key[e] > -np.inf), key=lambda e: (-key[e], e))[:K]
        ids[t, :len(order)] = order
        p, rel = _shares(z[t], ids[t], mode)
        gates[t] = scale * p
        tol[t] = np.abs(gates[t]) * (rel + 1) * U + 2.0 ** -126
    return ids, gates, tol


def route_backward(dgates, logits, ids, mode, scale=1.0):
    """(dlogits [T, E], bound) for given ids; an id outside [0, E) is no pick."""
    z, dg = np.asarray(logits, np.float64), np.asarray(dgates, np.float64)
    T, E = z.shape
    out, tol = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = (ids[t] >= 0) & (ids[t] < E)
        if not on.any():
            continue
        i = np.where(on, ids[t], -1)
        g = np.where(on, dg[t], 0.0)
        p, rel = _shares(z[t], i, mode)
        D = (p * g).sum()
        eD = ((rel + 8) * p * np.abs(g)).sum() * U          # four joins, a product and their roundings
        for k in np.flatnonzero(on):
            e = i[k]
            part = p[k] * g[k] if mode == "softmax_all" else p[k] * (g[k] - D)
            off = p[k] * ((rel[k] + 4) * (abs(g[k]) + abs(D)) * U + (0 if mode == "softmax_all" else eD))
            if mode == "sigmoid":
                s = 1 / (1 + np.exp(z[t, e]))
                part, off = part * s, off * s + abs(part) * s * 8 * U
            out[t, e] += scale * part
            tol[t, e] += abs(scale) * off
        if mode == "softmax_all":
            every, rel_all = _shares(z[t], np.arange(E), "softmax_all")
            out[t] -= scale * every * D
            tol[t] += abs(scale) * every * ((rel_all + 4) * abs(D) * U + eD)
        tol[t] += (np.abs(out[t]) + tol[t]) * (len(i) + 4) * U
    return out, tol + 2.0 ** -126


# -- rows ----------------------------------------------------------------------

def sort_pairs(topk, E):
    """(offsets [E + 1], dest like topk, pair [rows]) of a stable sort of the pairs by expert."""
    flat = np.asarray(topk).reshape(-1)
    dest, pair, offsets = np.full(len(flat), -1, np.int32), [], [0]
    for e in range(E):
        p = np.flatnonzero(flat == e)
        dest[p] = offsets[-1] + np.arange(len(p))
        pair += list(p)
        offsets.append(offsets[-1] + len(p))
    return np.array(offsets, np.int32), dest.reshape(np.shape(topk)), np.array(pair, np.int32)


def combine_backward(dest, y, gates, dout):
    """(dy rows by dest, dgates, bound of dgates) for dest [T, K], y [M, H], gates [T, K] or None, dout [T, H]."""
    y, dout = np.asarray(y, np.float64), np.asarray(dout, np.float64)
    T, K = dest.shape
    H = y.shape[1]
    dy, dg, tol = {}, np.zeros((T, K)), np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            r = dest[t, k]
            if r < 0:
                continue
            dy[int(r)] = (1.0 if gates is None else float(gates[t, k])) * dout[t]
            dg[t, k] = dout[t] @ y[r]
            # a lane's share of the row, the terms of a vector, and six joins
            tol[t, k] = (H / 64 + 18) * U * (np.abs(dout[t]) @ np.abs(y[r]))
    return dy, dg, tol


# -- 8 bits --------------------------------------------------------------------

def e4m3():
    """The 256 values: sign, 4 exponent bits (bias 7), 3 of mantissa; 0x7f and 0xff are NaN, there are no infinities."""
    v = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v[c] = np.nan if c & 127 == 127 else (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        if c & 128:
            v[c] = -v[c]
    return v


def _nearest(a):
    """Codes of values of at most 448: the nearest, halfway to the even one."""
    mag = e4m3()[:127]
    a = np.asarray(a, np.float64)
    hi = np.clip(np.searchsorted(mag, np.abs(a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = np.abs(np.abs(a) - mag[lo]), np.abs(mag[hi] - np.abs(a))
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (c | np.where(np.signbit(a), 128, 0)).astype(np.uint8)


def _power(top):
    """Exponents of the scales of blocks of these largest magnitudes (finite)."""
    top = np.asarray(top, np.float64)
    e = np.floor(np.log2(np.maximum(top, 2.0 ** -200))).astype(np.int64) - 8
    e = np.where(top > 448 * 2.0 ** e, e + 1, e)
    return np.maximum(np.where(top > 0, e, -126), -126)


def quantize_fp8(w):
    """w [Kin, N] -> codes [Kin, N] and scale bytes [kb, nb]; a block that is not finite: NaN codes, 127."""
    w = np.asarray(w, np.float64)
    Kin, N = w.shape
    kb, nb = -(-Kin // BLOCK), -(-N // BLOCK)
    codes, scales = np.zeros((Kin, N), np.uint8), np.zeros((kb, nb), np.uint8)
    for b in range(kb):
        for n in range(nb):
            at = np.s_[b * BLOCK:(b + 1) * BLOCK, n * BLOCK:(n + 1) * BLOCK]
            v = w[at]
            if not np.isfinite(v).all():
                codes[at], scales[b, n] = 127, 127
                continue
            e = int(_power(np.abs(v).max()))
            codes[at], scales[b, n] = _nearest(v / 2.0 ** e), e + 127
    return codes, scales


def pack_fp8(codes, scales):
    """The layout of the C header: (code bytes, scale bytes) of one matrix, flat."""
    Kin, N = codes.shape
    kb, nb = scales.shape
    cb = np.zeros((N // 32, kb, 8, 32, 16), np.uint8)
    for k in range(Kin):
        cb[:, k // 128, k % 128 // 16, :, k % 16] = codes[k].reshape(N // 32, 32)
    sb = np.full((nb, -(-kb // 4) * 4), 127, np.uint8)
    sb[:, :kb] = scales.T
    return cb.reshape(-1), sb.reshape(-1)


def fp8_values(codes, scales):
    """[Kin, N] float64 that codes and scales stand for."""
    Kin, N = codes.shape
    s = np.repeat(np.repeat(2.0 ** (scales.astype(np.float64) - 127), BLOCK, 0)[:Kin], BLOCK, 1)[:, :N]
    return e4m3()[codes] * s


def round_rows(a, off=None):
    """Rows [n, K] rounded to 8 bits, a scale for each 128; with `off`, how far the result may be from it if
    the values are off by that: a value may meet another code, or its block another scale."""
    a = np.asarray(a, np.float64)
    out, far = np.empty_like(a), np.zeros_like(a)
    table = e4m3()
    for k in range(0, a.shape[1], BLOCK):
        b = a[:, k:k + BLOCK]

        def at(v, e):
            return table[_nearest(np.clip(v / 2.0 ** e, -448, 448))] * 2.0 ** e

        e = _power(np.abs(b).max(1, keepdims=True))
        out[:, k:k + BLOCK] = at(b, e)
        if off is None:
            continue
        o = off[:, k:k + BLOCK]
        for e2 in (_power(np.maximum(np.abs(b) - o, 0).max(1, keepdims=True)), e,
                   _power((np.abs(b) + o).max(1, keepdims=True))):
            for v in (b - o, b + o):
                far[:, k:k + BLOCK] = np.maximum(far[:, k:k + BLOCK], np.abs(at(v, e2) - out[:, k:k + BLOCK]))
    return out if off is None else (out, far)


def fp8_ffn(x, topk, gates, w13, w2, unit=U, keep=0.0):
    """out [T, H] and a bound, elementwise, without the rounding of the output.  w13 [E, H, 2I], w2 [E, I, H]
    float64.  ``unit``: what the sum of a product may be off by, over its length times the sum of magnitudes,
    2^-24 for float32 sums; ``keep``: relative error of an expert's output where it is stored."""
    x, gates = np.asarray(x, np.float64), np.asarray(gates, np.float64)
    T, H = x.shape
    E, _, I2 = w13.shape
    I = I2 // 2
    xq = round_rows(x)
    out, off, mass = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    # float32 sums: each step one rounding; the matrix instruction's own: `unit` of the magnitudes as a whole
    span = (lambda n: n * U) if unit == U else (lambda n: n * U + unit)
    for t in range(T):
        for k, e in enumerate(topk[t]):
            if not 0 <= e < E:
                continue
            gu = xq[t] @ w13[e]
            dgu = span(H) * (np.abs(xq[t]) @ np.abs(w13[e]))
            g, v = gu[:I], gu[I:]
            s = g / (1 + np.exp(-g))
            a = s * v
            # |silu'| < 1.1; exponential, sum, quotient and product within 8 roundings
            da = 1.1 * dgu[:I] * (np.abs(v) + dgu[I:]) + np.abs(s) * dgu[I:] + np.abs(a) * 8 * U
            q, dq = (r[0] for r in round_rows(a[None], da[None]))
            y = q @ w2[e]
            dy = dq @ np.abs(w2[e]) + span(I) * ((np.abs(q) + dq) @ np.abs(w2[e]))
            # float16 with one power of two for 64: steps of 2^-24 where the largest is 2^14
            dy += keep * (np.abs(y) + dy) + (2.0 ** -38 * (np.abs(y) + dy).max() if keep else 0)
            out[t] += gates[t, k] * y
            off[t] += np.abs(gates[t, k]) * dy
            mass[t] += np.abs(gates[t, k]) * (np.abs(y) + dy)
    return out, off + (len(topk[0]) + 2) * U * mass
