"""fp64 CPU oracle of the rows' operators (include/qmm_rows.h) and of the
verification of drafts (include/qmv_verify.h). Inputs are numpy arrays of the
values (bf16 ones widened); test infrastructure only.
"""

from __future__ import annotations

import math

import numpy as np


def sort(ids, n_experts):
    """offsets, row_index, places of ids [tokens][top_k], one choice at a time."""
    ids = np.asarray(ids)
    tokens, top_k = ids.shape
    of = [[] for _ in range(n_experts)]
    for t in range(tokens):
        for j in range(top_k):
            if 0 <= ids[t, j] < n_experts:
                of[ids[t, j]].append((t, j))
    offsets = np.zeros(n_experts + 1, np.int32)
    row_index = np.full(tokens * top_k, -1, np.int32)
    places = np.full((tokens, top_k), -1, np.int32)
    row = 0
    for e in range(n_experts):
        for t, j in of[e]:
            row_index[row], places[t, j] = t, row
            row += 1
        offsets[e + 1] = row
    return offsets, row_index, places


def spread(x, places, out):
    out = np.array(out)
    for t, j in np.ndindex(*places.shape):
        if 0 <= places[t, j] < len(out):
            out[places[t, j]] = x[t]
    return out


def combine(z, places, w):
    """y and the sum of its terms' magnitudes, both [tokens][h]."""
    z = np.asarray(z, np.float64)
    y = np.zeros((len(places), z.shape[1]))
    mag = np.zeros_like(y)
    for t, j in np.ndindex(*places.shape):
        if 0 <= places[t, j] < len(z):
            term = z[places[t, j]] * (1.0 if w is None else float(w[t, j]))
            y[t] += term
            mag[t] += np.abs(term)
    return y, mag


def combine_grad(dy, z, places, w, dz):
    """dz (of the given one where no place names a row), dw, and dw's magnitudes."""
    dz = np.array(dz, np.float64)
    dy, z = np.asarray(dy, np.float64), np.asarray(z, np.float64)
    dw, mag = np.zeros(places.shape), np.zeros(places.shape)
    for t, j in np.ndindex(*places.shape):
        at = places[t, j]
        if 0 <= at < len(z):
            dz[at] = dy[t] * (1.0 if w is None else float(w[t, j]))
            dw[t, j] = math.fsum(dy[t] * z[at])
            mag[t, j] = np.abs(dy[t] * z[at]).sum()
    return dz, dw, mag


def lora(x, a, b, offsets, row_index, scale, ranks, base):
    """y and the magnitude of the sums behind what was added to it."""
    x, a, b = (np.asarray(v, np.float64) for v in (x, a, b))
    y = np.array(base, np.float64)
    mag = np.zeros_like(y)
    for e in range(len(a)):
        rank = a.shape[1] if ranks is None else min(max(int(ranks[e]), 0), a.shape[1])
        s = 1.0 if scale is None else float(scale[e])
        for r in range(offsets[e], offsets[e + 1]):
            row = r if row_index is None else row_index[r]
            if not 0 <= row < len(x):
                continue
            ae, be = a[e, :rank], b[e, :, :rank]
            y[row] += s * (be @ (ae @ x[row]))
            mag[row] += abs(s) * (np.abs(be) @ (np.abs(ae) @ np.abs(x[row])))
    return y, mag


def _weight(v):
    return float(v) if math.isfinite(v) and v > 0 else 0.0


def verify_one(p, q, drafts, u):
    """(accepted, the token that follows) of one request: p [drafts + 1][vocab], q likewise or None."""
    vocab = len(p[0])
    n = 0
    while n < len(drafts):
        d = int(drafts[n])
        if not 0 <= d < vocab:
            break
        if not float(u[n]) * (1.0 if q is None else float(q[n][d])) < float(p[n][d]):
            break
        n += 1
    left = [_weight(v) for v in p[n]]
    weights = left
    if n < len(drafts):
        if q is None:
            weights = [0.0 if i == drafts[n] else v for i, v in enumerate(left)]
        else:
            with np.errstate(invalid="ignore"):
                weights = [_weight(float(s) - float(t)) for s, t in zip(p[n], q[n])]
        if sum(weights) <= 0:
            weights = left
    total = math.fsum(weights)
    if total <= 0:
        return n, -1
    # from one on: the last weight, although a running sum may round above the whole
    target, run, last = float(u[-1]) * total if u[-1] < 1 else math.inf, 0.0, -1
    for i, v in enumerate(weights):
        if v > 0:
            run += v
            last = i
            if run > target:
                return n, i
    return n, last


def verify(p, q, drafts, lengths, u):
    requests, steps = len(p), len(p[0])
    accepted = np.zeros(requests, np.int32)
    out = np.full((requests, steps), -1, np.int32)
    for r in range(requests):
        have = steps - 1 if lengths is None else min(max(int(lengths[r]), 0), steps - 1)
        n, token = verify_one(p[r], None if q is None else q[r], drafts[r][:have], u[r])
        accepted[r] = n
        out[r, :n] = drafts[r][:n]
        out[r, n] = token
    return accepted, out
