"""Rows of seven chunks whose running sum, formed as the lanes of a wave form
it, is larger at a chunk without weight than at the one before it, and a total
of which half is the smaller of the two: for the tests of drawing. Plain
Python; nothing of it runs on a GPU.

A wave's inclusive scan adds the value 1, 2, 4, .. lanes before, so that lanes
4 and 5 of values w0 .. w5 have, with w5 = 0,
  ((w4 + w3) + (w2 + w1)) + w0   and   (w4 + (w3 + w2)) + (w1 + w0),
and a wave's sum of seven values (the others 0) is
  ((w0 + w1) + (w2 + w3)) + ((w4 + w5) + w6).
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

CHUNK = 4096                                   # elements of a row that are summed together


def scans(w):
    """The scan at lanes 4 and 5."""
    return ((w[4] + w[3]) + (w[2] + w[1])) + w[0], (w[4] + (w[3] + w[2])) + (w[1] + w[0])


def whole(w, last):
    return ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + 0.0) + last)


def last_for(w, total):
    """w6 such that the wave's sum is `total`, None where rounding leaves none."""
    guess = total - (((w[0] + w[1]) + (w[2] + w[3])) + w[4])
    for step in range(-4, 5):
        last = guess
        for _ in range(abs(step)):
            last = float(np.nextafter(last, np.inf if step > 0 else -np.inf))
        if whole(w, last) == total:
            return last
    return None


def below(v):
    """The largest fp32 number up to v."""
    a = np.float32(v)
    return float(a if float(a) <= v else np.nextafter(a, np.float32(-np.inf)))


def three(v):
    """A positive v as a sum of three fp32 numbers, exactly; none of them is negative."""
    a = below(v)
    b = below(v - a)
    c = below(v - a - b)
    assert (a + b) + c == v and c >= 0
    return a, b, c


def weights_row(seed):
    """Positive weights (fp32): row and the tokens that u = 1/2 may draw."""
    rng = np.random.default_rng(seed)
    while True:
        w = [float(x) for x in rng.uniform(0.1, 1.0, 5)]
        low, high = scans(w)
        last = last_for(w, 2 * low) if low < high else None
        if last is None or last <= 0:
            continue
        z = np.zeros(7 * CHUNK, np.float32)
        for c, v in [*enumerate(w), (6, last)]:
            z[c * CHUNK:c * CHUNK + 3] = three(v)
        return z, (4 * CHUNK, 4 * CHUNK + 1, 4 * CHUNK + 2, 6 * CHUNK)


def fma(a, b, c):
    return float(Fraction(a) * Fraction(b) + Fraction(c))


def exp2_taylor(t):
    """2^t for t <= 0 as the kernels form it: Taylor's polynomial of degree 12 about the nearest whole number."""
    c, v = [], 1.0
    for i in range(13):
        c.append(v)
        v = v * 0.69314718055994530941723212145818 / (i + 1)
    k = float(np.rint(t))
    p = c[12]
    for i in range(11, -1, -1):
        p = fma(p, t - k, c[i])
    return float(np.ldexp(p, int(k)))


def weight(logit):
    """Weight of a logit below the row's largest one, which is 0; temperature 1."""
    return exp2_taylor(float(logit) * 1.4426950408889634073599246810019)


def logit_for(w):
    """The fp32 logit whose weight comes nearest to w."""
    guess = np.float32(np.log(w))
    near = [guess]
    for way in (-np.inf, np.inf):
        x = guess
        for _ in range(3):
            x = np.nextafter(x, np.float32(way))
            near.append(x)
    return min((x for x in near if x <= 0), key=lambda x: abs(weight(x) - w))


def logits_row(seed):
    """The same for logits: weights of one token each, and in the last chunk those that make up its sum, the first
    one the row's largest."""
    rng = np.random.default_rng(seed)
    while True:
        z = np.full(7 * CHUNK, -np.inf, np.float32)
        at = [int(c * CHUNK) for c in range(5)]
        logits = [np.float32(x) for x in np.log(rng.uniform(0.3, 0.9, 5))]
        w = [weight(x) for x in logits]
        low, high = scans(w)
        last = last_for(w, 2 * low) if low < high else None
        if last is None or last <= 1:
            continue
        z[at] = logits
        z[6 * CHUNK] = 0.0
        total, places = 1.0, [6 * CHUNK + i for i in (1, 2, 3, 1024, 1025, 1026, 1027, 2048, 2049)]   # of the first lane, in its order
        for place in places:
            rest = last - total
            if rest <= 0:
                break
            x = logit_for(min(rest, 0.9))
            z[place] = x
            total += weight(x)
        if total == last:
            return z, (4 * CHUNK, 6 * CHUNK)
