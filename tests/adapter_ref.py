"""Low-rank adapters beside a shared projection in 64 bits, entry by entry,
from the definition in include/ep.h, and the bounds of the kernels.  numpy.

Bounds, with u = 2^-24 (fp32) and h = 2^-8 (bf16), half steps.  Products of
bf16 values are exact in fp32; a sum of n of them in any order is off by at
most 2 n u of the sum of their magnitudes (the factor 2 for the matrix
instructions, whose inner additions need not round to nearest).  scale * w *
(A_e x_t) has, besides the fp32 sum's error, three products (3u) and one
rounding to bf16 (`carried` = h of its value; two parts of bf16 leave h * h).
A result in bf16 is rounded once more.
Each quantity below comes with `mag`, the same sum over magnitudes.
"""
import numpy as np

U = 2.0 ** -24
H = 2.0 ** -8
TINY = 2.0 ** -120


def forward(x, W, a, b, idx, w, scale, carried=H):
    """-> out, bound, and what the backward needs."""
    T, K = idx.shape
    E = a.shape[0]
    D, r = x.shape[1], a.shape[1]
    coef = np.full((T, K), float(scale)) if w is None else scale * w.astype(np.float64)
    out, mag = x @ W.T, np.abs(x) @ np.abs(W).T
    bound = 2 * (D + r * K + 64) * U * mag
    saved = dict(coef=coef, entries=[])
    for t in range(T):
        by = {}
        for k in range(K):
            e = int(idx[t, k])
            if 0 <= e < E:
                by.setdefault(e, []).append(k)
        for e, ks in by.items():
            c = coef[t, ks].sum()
            cm = np.abs(coef[t, ks]).sum()
            u, um = a[e] @ x[t], np.abs(a[e]) @ np.abs(x[t])
            eu = 2 * D * U * um                                    # fp32 sum
            ec = abs(c) * eu + cm * (3 + len(ks)) * U * np.abs(u)     # times the coefficient
            ec = ec + carried * (np.abs(c * u) + ec)               # rounded to bf16
            out[t] += b[e] @ (c * u)
            bound[t] += np.abs(b[e]) @ (ec + 2 * (D + r * K + 64) * U * np.abs(c * u))
            saved["entries"].append((t, e, ks, c, cm, u, eu, ec))
    return out, bound + H * (np.abs(out) + bound) + TINY, saved


def backward(x, W, a, b, idx, w, scale, dy, saved, carried=H):
    """-> {name: (value, bound)} for dx, da, db, dw."""
    T, K = idx.shape
    E, r, D = a.shape
    O = W.shape[0]
    dx, dxb = dy @ W, 2 * (O + r * K + 64) * U * (np.abs(dy) @ np.abs(W))
    da, dab = np.zeros(a.shape), np.zeros(a.shape)
    db, dbb = np.zeros(b.shape), np.zeros(b.shape)
    dw, dwb = np.zeros((T, K)), np.zeros((T, K))
    n = 2 * (T + 64) * U
    for t, e, ks, c, cm, u, eu, ec in saved["entries"]:
        v, vm = b[e].T @ dy[t], np.abs(b[e]).T @ np.abs(dy[t])
        ev = 2 * O * U * vm
        evc = abs(c) * ev + cm * (3 + len(ks)) * U * np.abs(v)
        evc = evc + carried * (np.abs(c * v) + evc)
        dx[t] += a[e].T @ (c * v)
        dxb[t] += np.abs(a[e]).T @ (evc + 2 * (O + r * K + 64) * U * np.abs(c * v))
        da[e] += np.outer(c * v, x[t])
        dab[e] += np.outer(evc + n * (np.abs(c * v) + evc), np.abs(x[t]))
        db[e] += np.outer(dy[t], c * u)
        dbb[e] += np.outer(np.abs(dy[t]), ec + n * (np.abs(c * u) + ec))
        for k in ks:
            dw[t, k] = scale * (u * v).sum()
            dwb[t, k] = abs(scale) * ((np.abs(u) * ev + np.abs(v) * eu + eu * ev).sum() +
                                      2 * (r + 2) * U * np.abs(u * v).sum())
    rnd = lambda g, e: (g, e + H * (np.abs(g) + e) + TINY)  # noqa: E731
    return dict(dx=rnd(dx, dxb), da=rnd(da, dab), db=rnd(db, dbb), dw=(dw, dwb + TINY))
