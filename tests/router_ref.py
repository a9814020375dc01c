"""The router, the balance loss and their gradients in 64 bits, row by row,
from the definitions in include/ep.h; and the bounds the fp32 kernels are held
to.  numpy only.

Bounds, with u = 2^-24 (half a step of fp32).  A score is exp(z - m) or
1 / (1 + exp(-z)): the difference z - m is off by u |z - m|, which the
exponential turns into the same relative error, and the exponential itself by
4u; a score that is not 0 in fp32 has z - m > -104, so `spread` =
min(104, max z - min z) bounds the first part.  The sum over a row adds at most
64 + 6 terms one after the other (70u, for E = 4096; 4u less for its own scores'
share, which quotients cancel), its reciprocal 2u, a factor u each.  So a probability or a weight is
off by at most (spread + 80) u of its value; TINY covers scores that leave
the normal range of fp32.
  A gradient p (G - sum_j p_j G_j) has two such factors, products and the sum:
at most 2 (spread + 80) u + 70 u of p (|G| + sum_j p_j |G_j|).
"""
import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -120
BF16 = 2.0 ** -8          # half a step, relative


def clean(z):
    z = np.asarray(z, np.float64).copy()
    bad = np.isnan(z) | (z == np.inf)
    z[bad] = -np.inf
    return z, bad


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def scores(z, score):
    """Scores of a row up to a common factor, through their logarithms: the
    largest is 1, so that a quotient of them stands where all of them underflow
    (log sigmoid(z) = -log(1 + exp(-z)))."""
    live = z > -np.inf
    s = np.zeros_like(z)
    if not live.any():
        return s
    log = -np.logaddexp(0.0, -z[live]) if score == "sigmoid" else z[live]
    s[live] = np.exp(log - log.max())
    return s


def probs(z, score):
    s = scores(z, score)
    t = s.sum()
    return s / t if t > 0 else s


def route(z, K, score, bias=None, renorm=True, scale=1.0):
    """-> idx [T, K], w [T, K], bad [T]."""
    z, bad = clean(z)
    T, E = z.shape
    idx = np.full((T, K), -1, np.int32)
    w = np.zeros((T, K))
    for t in range(T):
        key = z[t].copy()
        if bias is not None:
            key = np.where(z[t] > -np.inf, sigmoid(z[t]) + bias.astype(np.float64), -np.inf)
            key[~np.isfinite(bias)] = -np.inf
        order = [e for e in np.argsort(-key, kind="stable")[:K] if key[e] > -np.inf]
        n = len(order)
        idx[t, :n] = order
        if n == 0:
            continue
        s = scores(z[t], score) if not renorm else scores(z[t][order], score)
        if renorm:
            w[t, :n] = scale * s / s.sum()
        elif score == "softmax":
            w[t, :n] = scale * (s / s.sum())[order]
        else:
            w[t, :n] = scale * sigmoid(z[t][order])
    return idx, w, bad.sum(axis=1).astype(np.int32)


def route_grad(z, idx, d_w, score, renorm, scale):
    """-> d_logits [T, E], and the size its rounding errors are relative to."""
    z, _ = clean(z)
    T, E = z.shape
    d, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = [(e, scale * float(g)) for e, g in zip(idx[t], d_w[t]) if 0 <= e < E and z[t, e] > -np.inf]
        if not on:
            continue
        es = np.array([e for e, _ in on])
        G = np.array([g for _, g in on])
        if renorm:
            s = scores(z[t][es], score)
            q = s / s.sum()
            slope = sigmoid(-z[t][es]) if score == "sigmoid" else 1.0
            np.add.at(d[t], es, q * (G - (q * G).sum()) * slope)
            np.add.at(size[t], es, q * (np.abs(G) + (q * np.abs(G)).sum()) * slope)
        elif score == "sigmoid":
            v = sigmoid(z[t][es]) * sigmoid(-z[t][es])
            np.add.at(d[t], es, G * v)
            np.add.at(size[t], es, np.abs(G) * v)
        else:
            p = probs(z[t], score)
            full, mag = np.zeros(E), np.zeros(E)
            np.add.at(full, es, G)
            np.add.at(mag, es, np.abs(G))
            d[t] = p * (full - (p * full).sum())
            size[t] = p * (mag + (p * mag).sum())
    return d, size


def balance(z, idx, score, coef=1.0, seq=None):
    """-> loss, counts [S, E], bad [2], and `grad(d_loss)` -> (d_logits, size)."""
    z, bad = clean(z)
    T, E = z.shape
    K = idx.shape[1]
    seq = [0, T] if seq is None else [int(v) for v in seq]
    S = len(seq) - 1
    counts = np.zeros((S, E), np.int32)
    live = (z > -np.inf).any(axis=1)
    P = np.stack([probs(z[t], score) for t in range(T)]) if T else np.zeros((0, E))
    total, n_live, bad_i, bad_z = 0.0, 0, 0, 0
    slopes = []
    for s in range(S):
        lo, hi = seq[s], seq[s + 1]
        e = idx[lo:hi].reshape(-1)
        counts[s] = np.bincount(e[(e >= 0) & (e < E)], minlength=E)
        bad_i += int(((e < -1) | (e >= E)).sum())
        bad_z += int(bad[lo:hi].sum())
        n = int(live[lo:hi].sum())
        f = E * counts[s] / (K * n) if n else np.zeros(E)
        slopes.append(f / n if n else f)
        n_live += n > 0
        if n:
            total += float((f * P[lo:hi].sum(axis=0)).sum()) / n
    per = 1.0 / n_live if n_live else 0.0

    def grad(d_loss):
        d, size = np.zeros((T, E)), np.zeros((T, E))
        for s in range(S):
            for t in range(seq[s], seq[s + 1]):
                p, f = P[t], slopes[s]
                dot = (p * f).sum()
                k = sigmoid(-z[t]) if score == "sigmoid" else 1.0
                k = np.where(z[t] > -np.inf, k, 0.0)
                d[t] = d_loss * coef * per * p * (f - dot) * k
                size[t] = abs(d_loss * coef * per) * p * (f + dot) * k
        return d, size

    return coef * total * per, counts, np.array([bad_i, bad_z], np.int32), grad


def spread(z):
    z, _ = clean(z)
    live = z[z > -np.inf]
    return min(104.0, float(live.max() - live.min())) if live.size else 0.0


def weight_bound(z):
    return (spread(z) + 80.0) * U


def grad_bound(z):
    return (2.0 * (spread(z) + 80.0) + 70.0) * U
