"""Adapters of small whole numbers: every sum that a kernel can form of them, in any order and over any parts of k, is a
whole number below 2^24, so fp32 holds each exactly and results have to be equal. |x| <= 2, |a|, |b| <= 1 and |scale| <= 2
keep |scale b a x| below 2 * 2 * 17408 * 128 < 2^23.1, and the base adds 8."""

import numpy as np

from oracle import rows_oracle as o

KS = [8, 64, 72, 200, 2048, 2056, 4096, 5120, 5128, 6144, 8192, 17408]
ROWS_RANKS = [(1, 8), (1, 16), (16, 16), (3, 24), (16, 32), (5, 40), (16, 64), (2, 128), (17, 16), (40, 32), (40, 64), (300, 16),
              (450, 72), (1600, 128)]
ADAPTERS = 3


def whole_numbers(rows, n, k, rank):
    g = np.random.default_rng((rows, n, k, rank))
    owner = g.integers(-1, ADAPTERS, rows)
    owner[0] = 0
    offsets, index, _ = o.sort(owner[:, None].astype(np.int32), ADAPTERS)
    return dict(x=g.integers(-2, 3, (rows, k)), a=g.integers(-1, 2, (ADAPTERS, rank, k)), b=g.integers(-1, 2, (ADAPTERS, n, rank)),
                scale=np.array([1, -2, 2], np.float32), ranks=np.array([rank, rank // 2 + 1, rank], np.int32),
                base=g.integers(-8, 9, (rows, n)), owner=owner, offsets=offsets, index=index)


def result(c, a=None):
    """base + scale b (a x) in fp64, where it is exact; a: another one than the case's."""
    a = c["a"] if a is None else a
    y = c["base"].astype(np.float64)
    for e in range(ADAPTERS):
        rows = np.flatnonzero(c["owner"] == e)
        used = c["ranks"][e]
        h = c["x"][rows].astype(np.float64) @ a[e, :used].astype(np.float64).T
        y[rows] += c["scale"][e] * (h @ c["b"][e, :, :used].astype(np.float64).T)
    return y


def by_block(c, row):
    """What each block of 64 of k adds to a row's results, [blocks][n]."""
    e, k = c["owner"][row], c["x"].shape[1]
    used, starts = c["ranks"][e], np.arange(0, k, 64)
    ax = c["a"][e, :used] * c["x"][row]
    return c["scale"][e] * (np.add.reduceat(ax, starts, axis=1).T @ c["b"][e, :, :used].T)
