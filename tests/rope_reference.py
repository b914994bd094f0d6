"""Plain 64-bit form of the rotary positions, with angles from exact rational
products, so that positions may be as far as int32 goes."""
import math
from fractions import Fraction

import numpy as np


def _inv_two_pi(bits=256):
    """floor(2^bits / 2 pi), by Machin's formula in integers."""
    one = 1 << (bits + 64)

    def atan_inv(n):
        term, total, k = one // n, one // n, 1
        while term:
            term = -(term // (n * n)) if term > 0 else (-term) // (n * n)
            k += 2
            total += term // k if term > 0 else -((-term) // k)
        return total
    pi = 4 * (4 * atan_inv(5) - atan_inv(239))
    return (one << bits) // (2 * pi)


_BITS = 256
_INV = _inv_two_pi(_BITS)


def turn_fraction(position, freq):
    """position * freq / 2 pi modulo 1 as a float in [-0.5, 0.5); freq: a float32."""
    f = Fraction(float(np.float32(freq))) * int(position)
    num = (f.numerator * _INV // f.denominator) % (1 << _BITS)
    if num >= 1 << (_BITS - 1):
        num -= 1 << _BITS
    return num / 2.0 ** _BITS if abs(num) < 1 << 1000 else 0.0


def cos_sin(positions, inv_freq, axis):
    """[rows, pairs] cosines and sines in 64 bits; positions int [n_axes, rows]."""
    known = {}
    t = np.empty((positions.shape[1], len(inv_freq)))
    for p, (f, a) in enumerate(zip(inv_freq, axis)):
        for r, pos in enumerate(positions[a].tolist()):
            key = (pos, float(f))
            if key not in known:
                known[key] = turn_fraction(pos, f)
            t[r, p] = known[key]
    return np.cos(2 * math.pi * t), np.sin(2 * math.pi * t)


def pairs_of(rot_dim, interleaved):
    i = np.arange(rot_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)


def turned(x, cos, sin, interleaved, scale=1.0, inverse=False):
    """x [rows, heads, D] in 64 bits; returns the turned rows and, per element, scale (|x| + |y|) of its pair."""
    a, b = pairs_of(2 * cos.shape[1], interleaved)
    c, s = cos[:, None], (-sin if inverse else sin)[:, None]
    out, mag = x.copy(), np.zeros_like(x)
    out[..., a] = scale * (x[..., a] * c - x[..., b] * s)
    out[..., b] = scale * (x[..., a] * s + x[..., b] * c)
    mag[..., a] = mag[..., b] = scale * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, mag
