"""Inputs and 64-bit results of attention with one leading key: head h scores
drops[h] with token 0, whose value is 0, and 0 with every other token."""
import math

import numpy as np

# Scores at which a probability exp(-drop) lies near the middle between two 16-bit numbers, where one rounding of it is
# off most.
DROPS = {"f16": (2.0625, 0.65625, 1.34375, 1.3115234375),
         "bf16": (1.359375, 0.62890625, 1.3671875, 1.3515625)}


def values(ps, d, seed):
    """Two pages of values between 0.5 and 1.5; token 0 of the first is 0."""
    v = 0.5 + np.random.default_rng(seed).random((2, ps, d))
    v[0, 0] = 0
    return v.astype(np.float32)


def expected(drops, seen, v):
    """out [heads][d] and lse [heads] of a query that sees `seen` tokens: page 0, then page 1 over and over."""
    ps = v.shape[1]
    whole, rest = divmod(max(0, seen - ps), ps)
    total = v[0, :min(ps, seen)].sum(0) + whole * v[1].sum(0) + v[1, :rest].sum(0)
    w = np.exp(-np.array(drops, np.float64))
    l = 1 + (seen - 1) * w
    return w[:, None] * total / l[:, None], np.array(drops) + np.log(l)


def STEPS_DECODE(n):
    """Longest chain of 32-bit additions of the single-token call: 64-token blocks shared by 304 CTAs at least, two
    products of 16 tokens a block and warp, then some 40 in the joins."""
    return 2 * (n // 64 // 304 + 1) + 40


def STEPS_PREFILL(n, cut):
    """The same of a chunk's call: products of 16 keys, the whole length or (cut into 64 pieces) a piece and the joins."""
    return n // 16 // 64 + 80 if cut else n // 16 + 16


def exponent_error(drops):
    """Relative error of a probability 2^-X, X = drop log2(e): the scale's product and constant and the difference are
    rounded to 32 bits (4 x 2^-24 X), the exponential to two steps."""
    x = np.abs(np.array(drops)) * math.log2(math.e)
    return math.log(2) * 4 * 2.0 ** -24 * x + 2.0 ** -22


def small_bounds(drops, n, steps, lost):
    """Relative error of out and error of lse, apart from the rounding of out: the probabilities' own, sums of `steps`
    terms in 32 bits (2^-23 each: the tensor pipe may truncate), two terms of 8 bits (bfloat16) at least, and `lost` of
    the largest probability for each key."""
    w = np.exp(-np.array(drops, np.float64))
    rel = 2 * (exponent_error(drops) + steps * 2.0 ** -23 + 2.0 ** -18) + lost / w
    # log2 of the sum and its product with ln 2, added to the maximum: 2^-22 of either
    return rel, exponent_error(drops) + steps * 2.0 ** -23 + 2.0 ** -21 * (np.abs(np.array(drops)) + math.log(n) + 1)


def two_term_bound(want, drops, n, eps):
    """Error of out where the probabilities enter as two 16-bit terms: (eps / 2)^2 of each, what 32 bits allow, and one
    rounding of out."""
    rel, _ = small_bounds(drops, n, STEPS_DECODE(n), 0.0)
    rel = rel - 2 * 2.0 ** -18 + 2 * (eps / 2) ** 2
    return np.abs(want) * (eps / 2 + rel[None, :, None]) + 2.0 ** -25
