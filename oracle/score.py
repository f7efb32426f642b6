"""Plain fp64 CPU oracle of the two other score functions over a block mask: a
learned relative position bias by buckets, and differential attention, with
their gradients.

TEST INFRASTRUCTURE ONLY, like the rest of this package: written from the
formulas, one head at a time, tokens in natural order, dense S x S matrices.
"""
from __future__ import annotations

import numpy as np

MASKED = -1e30  # a table entry at or below this masks its offsets


def coords(T, Hh, Ww):
    """(t, h, w) of every token, natural order."""
    p = np.arange(T * Hh * Ww)
    return p // (Hh * Ww), p // Ww % Hh, p % Ww


def token_mask(block_mask, T, Hh, Ww, tile):
    """[nb, nb] bool in block order -> [S, S] bool in natural token order."""
    pt, ph, pw = tile
    t, h, w = coords(T, Hh, Ww)
    b = ((t // pt) * (Hh // ph) + h // ph) * (Ww // pw) + w // pw
    return np.asarray(block_mask, bool)[np.ix_(b, b)]


def bias_matrix(table_row, bucket, T, Hh, Ww):
    """z's addend of every (query, key): three lookups by the offset key - query."""
    row = np.asarray(table_row, np.float64)
    row = np.where(row <= MASKED, -np.inf, row)
    S = T * Hh * Ww
    out, base = np.zeros((S, S)), 0
    for x, n in zip(coords(T, Hh, Ww), (T, Hh, Ww)):
        out += row[np.asarray(bucket)[base + (x[None, :] - x[:, None]) + n - 1]]
        base += 2 * n - 1
    return out


def softmax_rows(z, keep):
    """(P, log-sum-exp) over the kept keys; a row with none is 0 and -inf."""
    z = np.where(keep, z, -np.inf)
    m = z.max(1, keepdims=True)
    safe = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(z - safe)
    l = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(l[:, 0] > 0, safe[:, 0] + np.log(l[:, 0]), -np.inf)
    return e / np.where(l > 0, l, 1.0), lse


def bias_head(q, k, v, keep, bias):
    """(O, P, lse) of one head; keep, bias: [S, S]."""
    P, lse = softmax_rows(q @ k.T / np.sqrt(q.shape[1]) + bias, keep)
    return P @ v, P, lse


def bias_head_backward(q, k, v, g, P, O):
    """(dq, dk, dv, dS) of sum(O * g)."""
    s = 1.0 / np.sqrt(q.shape[1])
    dS = P * (g @ v.T - (g * O).sum(1, keepdims=True))
    return dS @ k * s, dS.T @ q * s, P.T @ g, dS


def bucket_sums(x, bucket, n_buckets, T, Hh, Ww):
    """Sum of x [S, S] over the pairs of every bucket, axis by axis."""
    out, base = np.zeros(n_buckets), 0
    for c, n in zip(coords(T, Hh, Ww), (T, Hh, Ww)):
        idx = np.asarray(bucket)[base + (c[None, :] - c[:, None]) + n - 1]
        out += np.bincount(idx.ravel(), weights=x.ravel(), minlength=n_buckets)
        base += 2 * n - 1
    return out


def diff_head(q, k, v, keep, lam):
    """(O, O2, [P1, P2], [lse1, lse2]) of one head."""
    e = q.shape[1] // 2
    P, lse = [], []
    for c in (slice(0, e), slice(e, 2 * e)):
        p, l = softmax_rows(q[:, c] @ k[:, c].T / np.sqrt(e), keep)
        P.append(p)
        lse.append(l)
    return (P[0] - lam * P[1]) @ v, P[1] @ v, P, lse


def diff_head_backward(q, k, v, g, P, lam):
    """(dq, dk, dv, dlam, [dS1, dS2]) of sum(O * g)."""
    e = q.shape[1] // 2
    s = 1.0 / np.sqrt(e)
    dP = g @ v.T
    dq, dk, dS = np.zeros_like(q), np.zeros_like(k), []
    for m, (c, w) in enumerate(((slice(0, e), 1.0), (slice(e, 2 * e), -lam))):
        D = (P[m] * dP).sum(1, keepdims=True)
        dS.append(w * P[m] * (dP - D))
        dq[:, c] = dS[m] @ k[:, c] * s
        dk[:, c] = dS[m].T @ q[:, c] * s
    return dq, dk, (P[0] - lam * P[1]).T @ g, -(P[1] * dP).sum(), dS
