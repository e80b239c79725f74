"""Head norms and position rotation in 64 bits for the tests, and the tolerance
they are held to.

A normed value is x inv g: the sum of D squares in fp32 is a sum of at most eight
in a row and five levels of pairs (13 roundings, half of them through the root),
then a division, an addition, a root, a division and two products: under 12
units of 2^-24.  An angle is rounded to fp32 within half a turn, pi 2^-24, cosine
and sine are within two units of 2^-24 times two, the two products and their
difference round once each.  So with a, b the pair's values
    |y - ref| <= 24 2^-24 (|a| + |b|),
plus half a step of the output's type.  A code of int8 stands within half of the
row's step, whose own error is that of the largest value."""
import numpy as np


def turned(x, gain, eps, pos, inv_freq, axis, interleaved):
    """x: T x heads x D, pos: axes x T; (values, the tolerance's |a| + |b|) in fp64."""
    x = np.array(x, np.float64)
    T, D, half = x.shape[0], x.shape[2], len(inv_freq)
    if gain is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    size = np.abs(x)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ax = 0 if axis is None else int(axis[i])
        t = pos[ax].astype(np.float64) * np.float64(inv_freq[i]) if 0 <= ax < len(pos) else np.zeros(T)
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        xa, xb = x[..., a].copy(), x[..., b].copy()
        x[..., a], x[..., b] = xa * c - xb * s, xb * c + xa * s
        size[..., a] = size[..., b] = np.abs(xa) + np.abs(xb)
    return x, size


def bound(ref, size, bf16):
    return 24 * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(ref) if bf16 else 0.0)


def code_bound(ref, size):
    step = np.abs(ref).max(-1, keepdims=True) / 127
    return step * (0.5 + 2.0 ** -12) + 24 * 2.0 ** -24 * size
