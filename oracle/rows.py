"""Row plan and per-request adapters (CPU oracle, numpy; adapters in float64).

Pins: the plan against a row-by-row construction, the adapters against a row-by-row loop.
"""

import numpy as np

TILE = 32


def plan(ids, n_ids):
    """(offsets, order, tiles) as the library lays them out."""
    ids = np.asarray(ids).reshape(-1)
    n = ids.size
    groups = [np.flatnonzero(ids == e) for e in range(n_ids)]
    offsets = np.concatenate([[0], np.cumsum([g.size for g in groups])]).astype(np.int32)
    order = np.full(n, -1, np.int32)
    kept = np.concatenate(groups) if n_ids else np.zeros(0)
    order[:kept.size] = kept
    tiles = np.zeros(((n + TILE - 1) // TILE + min(n, n_ids), 2), np.int32)
    tiles[:, 0] = -1
    at = 0
    for e, g in enumerate(groups):
        for f in range(0, g.size, TILE):
            tiles[at] = e, offsets[e] + f
            at += 1
    return offsets, order, tiles


def apply(X, A, B, ids, Y, scale=None, rows_per_x=1):
    """(y, bound terms P, |y0|) in float64 of Y[i] + scale[e] B[e] (A[e] X[i // rows_per_x])."""
    X, A, B, Y = (np.asarray(t, np.float64) for t in (X, A, B, Y))
    out, P = Y.copy(), np.zeros_like(Y)
    for e in range(A.shape[0]):
        rows = np.flatnonzero(np.asarray(ids) == e)
        x = X[rows // rows_per_x]
        s = 1.0 if scale is None else float(scale[e])
        out[rows] += s * (x @ A[e].T) @ B[e].T
        P[rows] = abs(s) * (np.abs(x) @ np.abs(A[e]).T) @ np.abs(B[e]).T
    return out, P, np.abs(Y)


def apply_bound(y, P, y0, K, r):
    """The stated bound of the library's fp32 accumulation and one bf16 rounding."""
    def gamma(n):
        return n * 2.0 ** -24 / (1 - n * 2.0 ** -24)
    return 2.0 ** -8 * np.abs(y) + (1 + 2.0 ** -8) * ((gamma(K + 12) + gamma(2 * r + 34) + 2.0 ** -17) * P
                                                     + gamma(2 * r + 34) * y0)
