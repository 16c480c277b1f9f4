"""Plain statements of the norm and rotation of queries and keys in 64 bits, with the bounds that 32-bit arithmetic and
one rounding at the end allow."""
from __future__ import annotations

import math

import numpy as np

UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4}
SMALLEST = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "e4m3": 2.0 ** -10}            # half the smallest step
LARGEST = 448.0


def frequencies(dim, scaling=0, base=10000.0, factor=1.0, low=0.0, high=0.0, original=0.0):
    f = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if scaling == 1:
        return [x / factor for x in f]
    if scaling == 2:
        out = []
        for x in f:
            wave = 2 * math.pi / x
            if wave < original / high:
                out.append(x)
            elif wave > original / low:
                out.append(x / factor)
            else:
                r = (original / wave - low) / (high - low)
                out.append((1 - r) * x / factor + r * x)
        return out
    if scaling == 3:
        low, high = low or 1.0, high or 32.0
        first = max(math.floor(dim * math.log(original / (high * 2 * math.pi)) / (2 * math.log(base))), 0)
        last = min(math.ceil(dim * math.log(original / (low * 2 * math.pi)) / (2 * math.log(base))), dim - 1)
        r = [min(1.0, max(0.0, (i - first) / (last - first if last > first else 1e-3))) for i in range(dim // 2)]
        return [x * (1 - t) + x / factor * t for x, t in zip(f, r)]
    return f


def rotated(x, weight, positions, freq, magnitude, begin, pairs, norm_dim, eps):
    """x [tokens][heads][dim] in 64 bits: (result, bound of a 32-bit computation's error before the last rounding)."""
    x = x.astype(np.float64)
    err = np.zeros_like(x)
    if weight is not None:
        n = norm_dim
        inverse = 1.0 / np.sqrt((x[..., :n] ** 2).sum(-1, keepdims=True) / n + eps)
        x = x.copy()
        x[..., :n] = x[..., :n] * inverse * weight.astype(np.float64)
        # n squares summed, half of that error through the root, which is 2 units (2^-22) off; eps, 1/n and three products 2^-24 each
        err[..., :n] = np.abs(x[..., :n]) * ((n / 2 + 6) * 2.0 ** -24 + 2.0 ** -22)
    d = 2 * len(freq)
    if d:
        angle = positions.astype(np.float64)[:, None, None] * np.asarray(freq)
        c, s = np.cos(angle) * magnitude, np.sin(angle) * magnitude
        part, perr = x[..., begin:begin + d], err[..., begin:begin + d]
        ia, ib = (np.arange(0, d, 2), np.arange(1, d, 2)) if pairs else (np.arange(d // 2), np.arange(d // 2) + d // 2)
        a, b = part[..., ia], part[..., ib]
        # a sine: its angle's conversion 2^-25 pi, the function 2^-23, the magnitude 2^-24: below 3 x 2^-23; two products and a sum
        # 2^-24 each of at most |a| + |b|
        e = magnitude * ((np.abs(a) + np.abs(b)) * (3 * 2.0 ** -23 + 3 * 2.0 ** -24) + perr[..., ia] + perr[..., ib])
        x, err = x.copy(), err.copy()
        part, perr = x[..., begin:begin + d], err[..., begin:begin + d]
        part[..., ia], part[..., ib] = a * c - b * s, b * c + a * s
        perr[..., ia] = perr[..., ib] = e
    return x, err


def stored(x, err, scale):
    """8-bit codes' values before their rounding: times 1 / scale in 32 bits, saturated."""
    y = x / scale
    return np.clip(y, -LARGEST, LARGEST), err / scale + np.abs(y) * 2.0 ** -23


def bound(x, err, kind):
    return UNIT[kind] * (np.abs(x) + err) + err + SMALLEST[kind]
