"""Oracle of the operators around the LM head (test infrastructure only):
float64 NumPy forms of the residual RMS norm and its gradients, the scaled
embedding lookup and its gradient, and the clipping by the global norm."""
from __future__ import annotations

import numpy as np


def _active(mask, R):
    return np.ones(R, bool) if mask is None else np.asarray(mask) != 0


def rmsnorm(x, weight, eps, residual=None, mask=None):
    """(y, s): s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight, zero on
    inactive rows.  Inactive rows are selected away, not multiplied."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    on = _active(mask, s.shape[0])
    y = np.zeros_like(s)
    a = s[on]
    y[on] = a / np.sqrt((a * a).mean(axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return y, s


def rmsnorm_grad(dy, s, weight, eps, ds=None, mask=None):
    """(dx, dweight) of sum(dy * y) + sum(ds * s)."""
    s = np.asarray(s, np.float64)
    w = np.asarray(weight, np.float64)
    on = _active(mask, s.shape[0])
    dx = np.zeros_like(s) if ds is None else np.array(ds, np.float64)
    a, d = s[on], np.asarray(dy, np.float64)[on]
    rms = np.sqrt((a * a).mean(axis=1, keepdims=True) + eps)
    n = a / rms
    dn = d * w
    dx[on] += (dn - n * (dn * n).mean(axis=1, keepdims=True)) / rms
    return dx, (d * n).sum(axis=0)


def embed(ids, table, scale):
    """scale * table[ids], zero rows for ids outside the table."""
    ids = np.asarray(ids)
    table = np.asarray(table, np.float64)
    out = np.zeros((ids.size, table.shape[1]))
    real = (ids >= 0) & (ids < table.shape[0])
    out[real] = scale * table[ids[real]]
    return out


def embed_grad(ids, dout, V, scale):
    """dweight[v] = scale * sum of dout[t] over ids[t] == v."""
    ids = np.asarray(ids)
    dout = np.asarray(dout, np.float64)
    dw = np.zeros((V, dout.shape[1]))
    for t in np.flatnonzero((ids >= 0) & (ids < V)):
        dw[ids[t]] += dout[t]
    return scale * dw


def clip_grads(grads, max_norm):
    """(norm, scaled gradients); nothing is scaled where the norm is not finite."""
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    c = min(1.0, max_norm / (norm + 1e-6)) if np.isfinite(norm) else 1.0
    return norm, [np.asarray(g, np.float64) * c for g in grads]
