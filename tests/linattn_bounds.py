"""How far fp32 work may be off the linear attention's exact values, in the norm.

An output is a sum of products whose partial sums have the size of the root of the terms' squares, A2 (terms of either
sign). A rounding is at most 2^-24 of what it rounds, and roundings go either way: n of them in a row are worth
sqrt(n) 2^-24 A2 in the norm. n: a sum over the channels of a score, one over the tokens of a chunk, one over the chunks,
and some 16 products, joins and splits. The powers of the decay are off by up to 2^-23 (the exponential) and 2^-24 (its
product with the scale): 4 x 2^-24 for their products with a term.
"""

import numpy as np

import oracle.linattn as O


def roundings(channels, T, C):
    return channels + C + -(-T // C) + 16


def bound(n):
    return (n ** 0.5 + 4) * 2.0 ** -24


def _sq(x):
    return None if x is None else x.double() ** 2


def forward_a2(q, k, v, ld, S0=None):
    """The roots of the sums of the terms' squares of o and S_T."""
    return [np.sqrt(t) for t in O.linattn_forward(_sq(q), _sq(k), _sq(v), 2 * ld.double(), _sq(S0))]


def backward_a2(q, k, v, ld, dO, S0=None, dS=None):
    m = O.linattn_backward(_sq(q), _sq(k), _sq(v), 2 * ld.double(), _sq(dO), _sq(S0), _sq(dS))
    return {n: np.sqrt(t) for n, t in m.items()}


def off(got, want, a2, heads_axis):
    """Largest norm of the error over the norm of A2, head by head (heads decay differently)."""
    e, m = np.moveaxis(np.asarray(got, np.float64) - want, heads_axis, 0), np.moveaxis(a2, heads_axis, 0)
    return max(float(np.linalg.norm(x) / np.linalg.norm(y)) for x, y in zip(e, m))
