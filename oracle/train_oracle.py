"""Plain CPU oracle of the norm in front of the layer, its gradients, the
gradients' 2-norm and the AdamW update with states in 32 or 8 bits, from the
formulas in ``include/moe.h``.

TEST INFRASTRUCTURE: shares no code with the HIP path and imports nothing from
it. Everything is float64 unless a function says otherwise; arrays are numpy.
"""
from __future__ import annotations

import math

import numpy as np

from .router_oracle import philox4x32

__all__ = ["norm", "norm_backward", "grad_norm", "adam_moments", "adam_update", "numbers", "code_values", "encode",
           "decode", "BLOCK"]

BLOCK = 128


def norm(s, w, b, kind, eps):
    """(y, mean, rstd) of rows s [T][d], one row at a time with exact sums."""
    T, d = s.shape
    y, mean, rstd = np.zeros((T, d)), np.zeros(T), np.zeros(T)
    for t in range(T):
        row = [float(v) for v in s[t]]
        if kind == "layer":
            mean[t] = math.fsum(row) / d
        e = s[t].astype(np.float64) - mean[t]
        rstd[t] = 1.0 / math.sqrt(math.fsum((v * v for v in e)) / d + eps)
        y[t] = e * rstd[t]
    if w is not None:
        y = y * w.astype(np.float64)
    if b is not None:
        y = y + b.astype(np.float64)
    return y, mean, rstd


def norm_backward(dy, s, w, kind, mean, rstd, dx_in=None):
    """(dx, dweight, dbias, and the absolute sums of dweight's and dbias's terms)."""
    dy, s = dy.astype(np.float64), s.astype(np.float64)
    h = (s - (mean[:, None] if kind == "layer" else 0.0)) * rstd[:, None]
    g = dy if w is None else dy * w.astype(np.float64)
    dx = g - h * (g * h).mean(axis=1, keepdims=True)
    if kind == "layer":
        dx = dx - g.mean(axis=1, keepdims=True)
    dx = dx * rstd[:, None]
    if dx_in is not None:
        dx = dx + dx_in.astype(np.float64)
    return dx, (dy * h).sum(axis=0), dy.sum(axis=0), np.abs(dy * h).sum(axis=0), np.abs(dy).sum(axis=0)


def grad_norm(grads, scale, max_norm):
    """(norm, factor) by exact sums."""
    n = abs(scale) * math.sqrt(math.fsum(float(v) ** 2 for g in grads for v in np.asarray(g).ravel()))
    return n, scale * min(1.0, max_norm / (n + 1e-6))


def adam_moments(g, gscale, m, v, beta1, beta2, dtype=np.float64):
    """The moments after a step; with dtype float32 every operation is rounded as the contract's order has it."""
    t = dtype
    x = g.astype(t) * t(gscale)
    b1, c1, b2, c2 = t(beta1), t(1.0 - beta1), t(beta2), t(1.0 - beta2)
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        return m.astype(t) * b1 + x * c1, v.astype(t) * b2 + (x * x) * c2


def adam_update(w, m, v, lr, step, beta1, beta2, eps, decay):
    """The weights after a step, from its moments."""
    w, m, v = (a.astype(np.float64) for a in (w, m, v))
    return w - lr / (1 - beta1 ** step) * m / (np.sqrt(v / (1 - beta2 ** step)) + eps) - lr * decay * w


def numbers(n, first, seed, offset):
    """The 16-bit numbers of elements first .. first + n - 1 of the list's numbering (first a multiple of 8)."""
    out = []
    for i in range(first // 8, (first + n + 7) // 8):
        words = philox4x32([i & 0xFFFFFFFF, i >> 32, offset & 0xFFFFFFFF, offset >> 32],
                           [seed & 0xFFFFFFFF, seed >> 32])
        for w in words:
            out += [w & 0xFFFF, w >> 16]
    return np.array(out[:n], np.int64)


def code_values(fraction):
    """What the magnitude codes of a scale of 2^0 stand for, ascending: gradual underflow below exponent 1."""
    out = []
    for c in range(16 << fraction):
        e, f = c >> fraction, (c & ((1 << fraction) - 1)) / (1 << fraction)
        out.append((1.0 + f) * 2.0 ** (e - 15) if e else f * 2.0 ** -14)
    return np.array(out)


def decode(code, scale, fraction):
    """float64 values of uint8 codes with a scale byte per BLOCK of them."""
    code = code.astype(np.int64)
    e = np.repeat(scale.astype(np.int64), BLOCK)[:code.size]
    table = code_values(fraction)
    if fraction == 3:
        val = np.where(code >= 128, -1.0, 1.0) * table[code & 127]
    else:
        val = table[code]
    return np.where(e == 255, np.nan, val * 2.0 ** (e - 127.0))


def encode(x, u, fraction):
    """(codes, scales) of fp32 values x: per block the least exponent whose top code holds the largest, then each
    value between two codes, away from zero where the part of a step and u / 2^16 reach 1."""
    table = code_values(fraction)
    n = x.size
    codes, scales = np.zeros(n, np.uint8), np.zeros(-(-n // BLOCK), np.uint8)
    for k in range(scales.size):
        at = slice(k * BLOCK, min(n, (k + 1) * BLOCK))
        b = x[at].astype(np.float64)
        a = np.abs(b)
        if not np.isfinite(a).all():
            scales[k] = 255
            continue
        e = 0
        top = a.max(initial=0.0)
        if top > 0:
            e = max(0, math.frexp(top)[1] - 1 + 127)
            if top > table[-1] * 2.0 ** (e - 127):
                e += 1
        if e >= 255:
            scales[k] = 255
            continue
        scales[k] = e
        a = a / 2.0 ** (e - 127)
        low = np.searchsorted(table, a, side="right") - 1
        step = np.where(low < table.size - 1, table[np.minimum(low + 1, table.size - 1)] - table[low], 1.0)
        # the part of a step, to fp32's grid at 2^-149 (the value as the code's exponents hold it)
        part = np.floor((a - table[low]) / step * 65536.0 + u[at])
        c = low + (part >= 65536)
        if fraction == 4:
            c = np.where((a > 0) & (c == 0), 1, c)
        else:
            c = c | np.where(np.signbit(b), 128, 0)
        codes[at] = c
    return codes, scales
