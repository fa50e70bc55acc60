"""Bounds of attention over the 4-bit cache, from the formats alone (test_kv4_formats checks on the CPU what
each format holds).

A rotated query block is three E2M3 parts.  Its largest magnitude comes to [3.75, 7.5); the last part's
step is 2^-11 at most there, so an element is off by 2^-12, QUERY = 2^-12 / 3.75 of the largest, and
independently of the others.  A score is off by |scale| QUERY max|q'| sum|k'| at most, and as a sum of
independent roundings by |scale| QUERY / sqrt(3) max|q'| |k'| in the mean square.

A weight p_j vs_j is three E4M3 parts where a sequence has few columns: the first leaves 2^-4 of it at
most, and each next one 2^-5 of what it gets (half a step of the largest number below a power of two),
WEIGHT_FEW = 2^-14, as long as the weight is 2^-14 of the tile's largest value scale.  Where it has many
columns it is rounded once to fp16, WEIGHT_MANY = 2^-11.  The sum of the weights is not rounded.  The
result is rounded to its type: 2^-11 or 2^-8 of itself.

Whole tensors, relative L2: the roundings are independent, each 1 / sqrt(3) of its largest in the mean
square; queries of size 1.5 and keys of size 1 put the scores' at 1.5e-4 (largest of 128 elements
about 4, |k| = 11.3, scale 128^-1/2; heads of 256 the same).
"""
import math

import numpy as np

QUERY = 2.0 ** -12 / 3.75
WEIGHT_FEW, WEIGHT_MANY = 2.0 ** -14, 2.0 ** -11
UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUMS = 2.0 ** -17  # fp32: sums of a few hundred terms, exponentials


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


def rel(dtype, few):
    w = WEIGHT_FEW if few else WEIGHT_MANY
    return math.sqrt((UNIT[dtype] ** 2 + w ** 2) / 3 + 1.5e-4 ** 2)


def blocks(x):
    return x.reshape(*x.shape[:-1], -1, 128)


def score_most(q, k, scale):
    """q [..., D], k [n, D], rotated: the most that any of the n scores is off, [...]."""
    top = np.abs(blocks(q)).max(-1)                   # [..., blocks]
    return abs(scale) * QUERY * (top @ np.abs(blocks(k)).sum(-1).T).max(-1)


def score_rms(q, k, scale):
    """The same in the mean square, of the longest of the keys."""
    top = np.abs(blocks(q)).max(-1)
    return abs(scale) * QUERY / math.sqrt(3) * np.sqrt((top ** 2) @ np.square(blocks(k)).sum(-1).T).max(-1)
