"""Plain 64-bit attention and cache rounding for the tests of the paged cache
and the attention over it, and the tolerances they are held to.

Tolerances.  A score s = scale sum_d q_d k_d is a sum of D fp32 products; with
A = max over keys of scale sum_d |q_d k_d| its error is taken as
    eps = 2^-21 sqrt(D) A + 2^-20
(eight units of fp32 rounding a term, errors adding as their square root, and
a few units for the exponential).  Errors of eps in every score change the
weights by e^eps at most, numerator and denominator both, so with V the
largest |v| seen
    |lse - ref| <= eps + 2^-20 |ref|,      |out - ref| <= 3 eps V,
plus, for a bf16 output, its rounding 2^-8 |ref|, and, where probabilities
enter the second product as bf16 (prompts), 2^-9 V.
"""
import math

import numpy as np


def bf16(x):
    """Values rounded to nearest-even bfloat16 (finite input)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return r.view(np.float32)


def quantise(x):
    """int8 codes and fp32 scales of the rows (last axis) of an fp32 array."""
    x = np.asarray(x, np.float32)
    s = np.abs(x).max(-1) / np.float32(127)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s[..., None] > 0, np.rint(x / s[..., None]), 0)
    return c.astype(np.int8), s.astype(np.float32)


def attend(q, k, v, scale, seen=None):
    """q: queries x D, k, v: keys x D, seen: queries x keys; (out, lse, eps, V)."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    nq, D = q.shape
    out, lse, eps = np.zeros((nq, D)), np.full(nq, -math.inf), np.zeros(nq)
    big = np.zeros(nq)
    for i in range(nq):
        use = np.arange(len(k)) if seen is None else np.flatnonzero(seen[i])
        if len(use) == 0:
            continue
        s = scale * (k[use] @ q[i])
        m = s.max()
        p = np.exp(s - m)
        out[i], lse[i] = p @ v[use] / p.sum(), m + math.log(p.sum())
        A = scale * (np.abs(k[use]) @ np.abs(q[i])).max()
        eps[i] = 2.0 ** -21 * math.sqrt(D) * A + 2.0 ** -20
        big[i] = np.abs(v[use]).max()
    return out, lse, eps, big


def check(out, lse, ref, bf16_out, bf16_p, what=""):
    """Holds out (queries x D) and lse (queries, or None) to attend()'s result."""
    o, l, eps, big = ref
    out = np.asarray(out, np.float64)
    bound = (3 * eps * big)[:, None] + np.zeros_like(o)
    if bf16_out:
        bound = bound + 2.0 ** -8 * np.abs(o)
    if bf16_p:
        bound = bound + (2.0 ** -9 * big)[:, None]
    assert np.isfinite(out).all(), f"{what}: non-finite output"
    err = np.abs(out - o)
    i = np.unravel_index(np.argmax(err - bound), err.shape) if err.size else None
    assert (err <= bound).all(), f"{what}: at {i} {out[i]} for {o[i]}, bound {bound[i]:.3e}"
    if lse is not None:
        lse = np.asarray(lse, np.float64)
        none = np.isneginf(l)
        assert (np.isneginf(lse) == none).all(), f"{what}: lse of empty rows"
        d = np.abs(lse[~none] - l[~none])
        assert (d <= eps[~none] + 2.0 ** -20 * np.abs(l[~none])).all(), f"{what}: lse off by {d.max():.3e}"
