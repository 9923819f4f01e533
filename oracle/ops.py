"""Oracle of the operators around the LM head (test infrastructure only):
float64 NumPy forms of the residual RMS norm and its gradients, the scaled
embedding lookup and its gradient, the clipping by the global norm, the scores of logits and
their gradient, and the orthogonalised update."""
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


def token_scores(x, tokens=None, k=0, scale=1.0, mask=None):
    """(logprob [N, M], entropy, lse, top_logprob [N, k], top_ids [N, k]) of
    softmax(scale x), row by row.  tokens [N, M]; -1 and others outside: 0.
    Inactive rows: zeros, ids -1."""
    x = np.asarray(x, np.float64)
    N, V = x.shape
    tokens = np.full((N, 0), -1) if tokens is None else np.asarray(tokens)
    on = _active(mask, N)
    lp, ent, lse = np.zeros(tokens.shape), np.zeros(N), np.zeros(N)
    top, ids = np.zeros((N, k)), np.full((N, k), -1)
    for i in np.flatnonzero(on):
        z = scale * x[i]
        rank = np.where(np.isnan(z), np.inf, z + 0.0)
        # NaN above +inf, then value, then column
        order = np.lexsort((np.arange(V), -rank, ~np.isnan(z)))[:k]
        ids[i] = order
        if np.isnan(z).any() or np.isposinf(z).any() or np.isneginf(z).all():
            lse[i] = ent[i] = np.nan
            logp = np.full(V, np.nan)
        else:
            d = z - z.max()                 # first: z may be as large as its type allows
            s = np.log(np.exp(d).sum())
            lse[i], logp = z.max() + s, d - s
            real = np.maximum(d, -1e4)      # 0 * -inf counts as 0
            ent[i] = s - (np.exp(real - s) * real).sum()
        top[i] = logp[order]
        for j, t in enumerate(tokens[i]):
            if 0 <= t < V:
                lp[i, j] = logp[t]
    return lp, ent, lse, top, ids


def token_scores_grad(g_lp, g_ent, x, tokens, lse, entropy, scale=1.0, mask=None):
    """Gradient of sum(g_lp * logprob) + sum(g_ent * entropy) at x."""
    x = np.asarray(x, np.float64)
    N, V = x.shape
    dx = np.zeros((N, V))
    for i in np.flatnonzero(_active(mask, N)):
        z = scale * x[i]
        p = np.exp(z - lse[i])
        logp = np.where(p > 0, z - lse[i], 0.0)
        real = [(j, t) for j, t in enumerate(tokens[i] if tokens is not None else []) if 0 <= t < V]
        dx[i] = -p * sum(g_lp[i][j] for j, _ in real)
        if g_ent is not None:
            dx[i] -= p * g_ent[i] * (logp + entropy[i])
        for j, t in real:
            dx[i, t] += g_lp[i][j]
        dx[i] *= scale
    return dx


def orthogonalize(g, coeffs, eps):
    """Newton-Schulz products of one matrix: x = g / (|g| + eps), then
    x = a x + (b q + c q q) x, q = x x', for each (a, b, c) of coeffs."""
    x = np.asarray(g, np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for a, b, c in coeffs:
        q = x @ x.T
        x = a * x + (b * q + c * (q @ q)) @ x
    return x.T if tall else x


def momentum_update(g, momentum, beta, nesterov):
    """(new momentum, update): m' = beta m + (1 - beta) g, the update m' or with
    nesterov beta m' + (1 - beta) g."""
    g = np.asarray(g, np.float64)
    m = beta * np.asarray(momentum, np.float64) + (1 - beta) * g
    return m, beta * m + (1 - beta) * g if nesterov else m
