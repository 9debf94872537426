"""A tight measure of the delta rule's results, one number per output: the 2-norm of the error over the 2-norm of the values.

Bounds per element take every error at its worst and in the same place; most values are far below them. Over all of a result the
errors of a float32 evaluation, independent in sign, add up in quadrature: a sum of n terms is off by sqrt(n) roundings of 2^-24
of what it adds up, n = dk + dv + 64 for the longest sum of a token's step. What a sum adds up is a few times its value here (keys and queries of
norm 1, beta at most 1), and a result is behind a few such sums: 4 sqrt(n) 2^-24 in all, 4.3e-6 at 128 columns. A bfloat16 result is rounded
once more, by at most 2^-8 of every value. A factor held in 16 bits instead of 24 (2^-17 per value, in every step), a dropped term or a
gradient of zeros are past that."""

import numpy as np

OUTPUTS = ("o", "last", "dq", "dk", "dv", "dg", "dbeta", "dstate")
ROUNDED = ("o", "dq", "dk", "dv")   # to the inputs' type

SHAPES = [(2, 65, 2, 1, 120, 120), (1, 130, 3, 3, 9, 33), (1, 200, 4, 2, 64, 72), (2, 127, 2, 1, 65, 17), (1, 191, 1, 1, 128, 128), (1, 300, 1, 1, 16, 7)]
SEGMENTED = [(1, 700, 1, 1, 48, 40), (1, 1090, 2, 1, 128, 128), (1, 1600, 1, 1, 100, 33)]


def bound(name, dk, dv, bf):
    return 4 * np.sqrt(dk + dv + 64) * 2.0 ** -24 + (2.0 ** -8 if bf and name in ROUNDED else 0.0)


def error(got, want):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    return float(np.sqrt(((got - want) ** 2).sum() / (want ** 2).sum()))


def check(name, got, want, dk, dv, bf):
    e, b = error(got, want), bound(name, dk, dv, bf)
    assert e <= b, "%s: off by %.3g, %.3g of its bound" % (name, e, e / b)
