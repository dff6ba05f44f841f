"""Plain 64-bit attention by its definition, token by token, for the GPU tests of the
differential and the windowed attention, with an elementwise bound of the kernels' rounding.

The bound.  A kernel's weighted sum of V rounds every probability once to binary16 (relative
2^-11, half a step) and keeps scores, sums and statistics in binary32.  A probability below
binary16's normal range is off by at most 2^-25, against a row maximum of at least 1.  Scores in
binary32 (products exact, sums of d terms) and exp2 leave a relative error of at most
2^-16 here (|score| < 2^5).  So an output row O = A V is off by at most
    E = (2^-11 + 2^-16) A|V| + n 2^-25 max|V|.
The final rounding to binary16 adds 2^-11 of the value, or 2^-25.
"""
import numpy as np

U16 = 2.0 ** -11


def f64(bits):
    return np.asarray(bits).view(np.float16).astype(np.float64)


def rows_of(pool, row, lo, hi, P, g):
    """Positions [lo, hi) of KV head g through a table row, as float64 [hi - lo][d]."""
    pos = np.arange(lo, hi)
    return f64(np.ascontiguousarray(pool[row[pos // P], g, pos % P]))


def weighted(q, K, V, scale, sink=None):
    """(A V, E) for queries q [G][e] over K [n][e], V [n][d]; sink [G] joins the denominator."""
    x = scale * (q @ K.T)
    m = x.max(1, keepdims=True)
    w = np.exp(x - m)
    den = w.sum(1, keepdims=True)
    if sink is not None:
        with np.errstate(over="ignore"):
            den = den + np.exp(np.asarray(sink, np.float64)[:, None] - m)
    A = w / den
    E = (U16 + 2.0 ** -16) * (A @ np.abs(V)) + (1 / den) * len(K) * 2.0 ** -25 * np.abs(V).max()
    return A @ V, E


def _rounded(out, E):
    return out, E * 1.05 + U16 * np.abs(out) + 2.0 ** -25


def diff_attention(q, kp, vp, tpt, kv, scale, lam, w=None, eps=1e-5, out_scale=1.0):
    """Differential attention [T][Hq][d] and its error bound."""
    q, lam = f64(q), np.asarray(lam, np.float64)
    T, Hq, d = q.shape
    _, Hkv, P, _ = kp.shape
    G, e = Hq // Hkv, d // 2
    out, tol = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    for t in range(T):
        if kv[t] <= 0:
            continue
        for g in range(Hkv):
            K, V = (rows_of(p, tpt[t], 0, kv[t], P, g) for p in (kp, vp))
            h = slice(g * G, (g + 1) * G)
            (o1, e1), (o2, e2) = (weighted(q[t, h, i:i + e], K[:, i:i + e], V, scale)
                                  for i in (0, e))
            la = lam[h, None]
            y, E = o1 - la * o2, e1 + np.abs(la) * e2
            if w is not None:
                f = 1 / np.sqrt((y ** 2).mean(1, keepdims=True) + eps)
                # d(y f) <= f E + |y| f^2 d(rms), d(rms) <= the root mean square of E
                E = f * E + np.abs(y) * f ** 2 * np.sqrt((E ** 2).mean(1, keepdims=True))
                y, E = y * f * np.asarray(w, np.float64), E * np.abs(np.asarray(w, np.float64))
            out[t, h], tol[t, h] = _rounded(y * out_scale, E * abs(out_scale))
    return out, tol


def window_attention(q, kp, vp, tpt, kv, scale, window, sink=None):
    """Windowed attention [T][Hq][d] and its error bound."""
    q = f64(q)
    T, Hq, d = q.shape
    _, Hkv, P, _ = kp.shape
    G = Hq // Hkv
    out, tol = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    for t in range(T):
        if kv[t] <= 0:
            continue
        lo = max(0, int(kv[t]) - window)
        for g in range(Hkv):
            K, V = (rows_of(p, tpt[t], lo, kv[t], P, g) for p in (kp, vp))
            h = slice(g * G, (g + 1) * G)
            o, E = weighted(q[t, h], K, V, scale, None if sink is None else sink[h])
            out[t, h], tol[t, h] = _rounded(o, E)
    return out, tol


def assert_within(got, ref, tol, what=""):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    bad = np.abs(got - ref) > tol
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of bounds; first {i}: "
                             f"{got[i]} for {ref[i]} +- {tol[i]}")
