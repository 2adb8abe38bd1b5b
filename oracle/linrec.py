"""fp64 elementwise gated linear recurrence and its gradients, token by token.

Test infrastructure, like the rest of this package.  Pinned in
``tests/test_oracle_linrec.py`` by closed forms (constant gates, a forgetting
gate) and the gradients by differences.
"""
import numpy as np


def replay(x, g, cu, h0=None):
    """(y [T, D], s [N, D]) of h_t = exp(g_t) h_{t-1} + x_t for every packed sequence."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    y = np.zeros_like(x)
    s = np.zeros((len(cu) - 1, x.shape[1]))
    for n in range(len(cu) - 1):
        h = np.zeros(x.shape[1]) if h0 is None else np.asarray(h0[n], np.float64)
        for t in range(cu[n], cu[n + 1]):
            h = np.exp(g[t]) * h + x[t]
            y[t] = h
        s[n] = h
    return y, s


def backward(g, y, dy, cu, h0=None, ds=None):
    """(dx, dg, dh0), with h_{t-1} taken from y."""
    g, y, dy = (np.asarray(a, np.float64) for a in (g, y, dy))
    dx, dg = np.zeros_like(y), np.zeros_like(y)
    dh0 = np.zeros((len(cu) - 1, y.shape[1]))
    for n in range(len(cu) - 1):
        p = np.zeros(y.shape[1]) if ds is None else np.asarray(ds[n], np.float64)
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            before = y[t - 1] if t > cu[n] else (0.0 if h0 is None else np.asarray(h0[n], np.float64))
            dx[t] = dy[t] + p
            p = np.exp(g[t]) * dx[t]
            dg[t] = p * before
        dh0[n] = p
    return dx, dg, dh0
