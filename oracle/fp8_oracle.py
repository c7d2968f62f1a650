"""CPU fp64 oracle of the e4m3 and grouped products -- test infrastructure only.

Written from the definitions: the e4m3 format bit by bit, rounding on a table of
its values, products in fp64. Nothing here comes from the kernels' code.
"""

from __future__ import annotations

import numpy as np

MAX = 448.0
TINY = 2.0 ** -126
BLOCK = 128


def e4m3_values() -> np.ndarray:
    """The values of the 256 codes: (-1)^s 2^(e-7) (1 + m/8), subnormals (-1)^s 2^-6 m/8, 0x7F and 0xFF NaN."""
    out = np.empty(256)
    for code in range(256):
        s, e, m = code >> 7, (code >> 3) & 15, code & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = np.nan
        out[code] = -v if s else v
    return out


VALUES = e4m3_values()


def decode(codes) -> np.ndarray:
    return VALUES[np.asarray(codes, dtype=np.uint8)]


def encode(v) -> np.ndarray:
    """Nearest e4m3 code of finite v (clamped to 448), ties to the even mantissa; signed zeros keep their sign."""
    v = np.asarray(v, dtype=np.float64)
    grid = VALUES[:127]                                     # non-negative finite values in code order
    a = np.minimum(np.abs(v), MAX)
    hi = np.searchsorted(grid, a, side="left")              # first value >= a
    lo = np.maximum(hi - 1, 0)
    down, up = a - grid[lo], grid[hi] - a
    code = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def blocks(k: int) -> int:
    return -(-k // BLOCK)


def quant(x):
    """(codes [m, k], scales fp32 [blocks, m]) of finite fp32/bf16-valued rows x [m, k]."""
    x = np.asarray(x, dtype=np.float64)
    m, k = x.shape
    codes = np.empty((m, k), dtype=np.uint8)
    scales = np.empty((blocks(k), m), dtype=np.float32)
    for b in range(blocks(k)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        s = np.maximum((np.abs(part).max(1) / MAX).astype(np.float32), np.float32(TINY))
        scales[b] = s
        quotient = (part / s.astype(np.float64)[:, None]).astype(np.float32)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = encode(quotient)
    return codes, scales


def silu_mul(x):
    """silu(gate) * up in fp64 of rows [m, 2 k]."""
    x = np.asarray(x, dtype=np.float64)
    k = x.shape[1] // 2
    gate, up = x[:, :k], x[:, k:]
    with np.errstate(over="ignore"):
        return gate / (1 + np.exp(-gate)) * up


def rows_f64(codes, scales) -> np.ndarray:
    k = codes.shape[1]
    return decode(codes) * np.repeat(np.asarray(scales, dtype=np.float64).T, BLOCK, axis=1)[:, :k]


def weights_f64(codes, scales) -> np.ndarray:
    n, k = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, dtype=np.float64), BLOCK, axis=0)[:n], BLOCK, axis=1)[:, :k]
    return decode(codes) * s


def product(x, w):
    """(y, sum |x w|) in fp64 of dense rows x [m, k] and w [n, k]."""
    with np.errstate(invalid="ignore"):
        return x @ w.T, np.abs(x) @ np.abs(w).T


def grouped(x, w, offsets, y, index=None):
    """Grouped product into a copy of y (fp64), and the sums of magnitudes; w is a list of [n, k] matrices."""
    y = np.array(y, dtype=np.float64)
    mag = np.zeros_like(y)
    for e, we in enumerate(w):
        run = np.arange(offsets[e], offsets[e + 1])
        src = run if index is None else np.asarray(index)[run]
        inside = (src >= 0) & (src < len(x))
        y[run], mag[run] = 0.0, 0.0
        if inside.any():
            y[run[inside]], mag[run[inside]] = product(x[src[inside]], we)
    return y, mag
