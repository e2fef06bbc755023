"""Softmax rows over the 8-bit caches in float64, and what rounding may do to them."""
import math

import numpy as np

from block_util import D, U16


def rows_of(q, K, V, hid=None):
    """Rows q [n][D] over K, V [L][D] in float64: weights, outputs, largest |q| . |k| / sqrt D."""
    s = q @ K.T / math.sqrt(D)
    mag = np.abs(q) @ np.abs(K).T / math.sqrt(D)
    if hid is not None:
        s, mag = np.where(hid, -np.inf, s), np.where(hid, 0.0, mag)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    return p, p @ V, mag.max(1, keepdims=True)


def variance(p, V, ref):
    """Of an output's error: a weight and the output are rounded to fp16 once each.  The error of a
    rounding is spread evenly over +- half a step, at most U16 of the value: U16^2 / 3 of its
    square; below fp16's normal numbers the output's step is 2^-24.  Weights' errors are independent."""
    return U16 ** 2 / 3 * ((p * p) @ (V * V) + ref * ref) + 2.0 ** -48 / 12


def worst(p, V, ref, mag):
    """What an element's error is at most: weights U16 of their products each, fp32 scores and sums
    (2^-24 of the magnitudes for each of 128 products, in numerator and denominator; 2^-19 for
    the exponential and the sums over tiles), the output's rounding."""
    ds = mag * 128 * 2.0 ** -24 + 2.0 ** -20
    return (p @ np.abs(V)) * (2 * ds + 1.1 * U16 + 2.0 ** -19) + U16 * np.abs(ref) + 2.0 ** -25


class Errors:
    """Squares of errors against their variances, over many outputs."""
    def __init__(self):
        self.err, self.var = 0.0, 0.0

    def add(self, got, q, K, V, hid=None):
        p, ref, mag = rows_of(q, K, V, hid)
        err = np.abs(got - ref)
        assert np.all(err <= worst(p, V, ref, mag)), (err / worst(p, V, ref, mag)).max()
        self.err += (err ** 2).sum()
        self.var += variance(p, V, ref).sum()
        return p

    def check(self):
        # the variances are upper bounds (half of them for evenly spread mantissas); thousands of
        # outputs, whose weights are a row's, leave 20% of room
        assert self.err <= 1.2 * self.var, "error %.3g times what roundings give" % math.sqrt(self.err / self.var)
