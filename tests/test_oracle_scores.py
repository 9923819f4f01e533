"""Pins of the oracle of the scores of logits and of the orthogonalised update:
closed forms, scipy, central differences, torch (CPU only)."""
import numpy as np
import pytest
import torch
from scipy.special import log_softmax
from scipy.stats import entropy as scipy_entropy

import oracle


def logits(N, V, seed=0):
    return np.random.default_rng(seed).normal(size=(N, V)) * 2


@pytest.mark.parametrize("scale", [1.0, 0.5, 3.0])
def test_forward_against_scipy(scale):
    x = logits(5, 40)
    t = np.random.default_rng(1).integers(0, 40, (5, 3))
    lp, ent, lse, top, ids = oracle.token_scores(x, t, 7, scale)
    ref = log_softmax(scale * x, axis=1)
    assert np.allclose(lp, np.take_along_axis(ref, t, 1), atol=1e-12)
    assert np.allclose(ent, scipy_entropy(np.exp(ref), axis=1), atol=1e-12)
    assert np.allclose(lse, np.logaddexp.reduce(scale * x, axis=1), atol=1e-12)
    assert np.allclose(top, np.sort(ref, axis=1)[:, ::-1][:, :7], atol=1e-12)
    assert np.array_equal(ids, np.argsort(-x, axis=1, kind="stable")[:, :7])


def test_forward_special_rows():
    inf, nan = np.inf, np.nan
    x = np.array([[1.0, 1.0, 1.0, 1.0], [-inf, 2.0, -inf, -inf], [-inf] * 4, [0.0, nan, 9.0, -0.0],
                  [0.0, -0.0, inf, 0.0], [5.0, 6.0, 7.0, 8.0]])
    lp, ent, lse, top, ids = oracle.token_scores(x, [[0, -1, 4]] * 6, 3, mask=[1, 1, 1, 1, 1, 0])
    assert np.allclose(ent[:2], [np.log(4), 0]) and np.allclose(lse[:2], [1 + np.log(4), 2])
    assert np.isnan(ent[2:5]).all() and np.isnan(lse[2:5]).all() and np.isnan(lp[2:5, 0]).all()
    assert lp[1, 0] == -inf and (lp[:, 1:] == 0).all()
    assert ids.tolist() == [[0, 1, 2], [1, 0, 2], [0, 1, 2], [1, 2, 0], [2, 0, 1], [-1] * 3]
    assert (lp[5] == 0).all() and ent[5] == lse[5] == 0 and (top[5] == 0).all()


def test_gradient_against_differences():
    x, scale, h = logits(3, 9, 2), 0.7, 1e-5
    t = np.array([[1, 1, -1], [0, 8, 3], [-1, -1, -1]])
    g = np.random.default_rng(3).normal(size=(3, 3))
    ge = np.array([0.3, -1.1, 0.8])
    mask = [1, 1, 1]

    def loss(x):
        lp, ent, *_ = oracle.token_scores(x, t, 0, scale, mask)
        return (g * lp).sum() + (ge * ent).sum()

    _, ent, lse, _, _ = oracle.token_scores(x, t, 0, scale, mask)
    dx = oracle.token_scores_grad(g, ge, x, t, lse, ent, scale, mask)
    for i in range(3):
        for v in range(9):
            d = np.zeros_like(x)
            d[i, v] = h
            assert abs((loss(x + d) - loss(x - d)) / (2 * h) - dx[i, v]) < 1e-8
    off = oracle.token_scores_grad(g, None, x, t, lse, ent, scale, [0, 1, 0])
    assert (off[[0, 2]] == 0).all() and np.allclose(off[1].sum(), 0)


def test_gradient_where_tokens_cannot_be():
    x = logits(1, 6)
    x[0, 2] = -np.inf
    _, ent, lse, _, _ = oracle.token_scores(x)
    dx = oracle.token_scores_grad([[0.5]], [1.0], x, [[1]], lse, ent)
    assert np.isfinite(dx).all() and dx[0, 2] == 0


@pytest.mark.parametrize("n,m", [(6, 9), (9, 6), (5, 5), (1, 4)])
def test_orthogonalize_on_singular_values(n, m):
    """Each step is the odd polynomial a s + b s^3 + c s^5 of the singular values."""
    g = np.random.default_rng(n * m).normal(size=(n, m))
    coeffs = [(3.4445, -4.7750, 2.0315)] * 3 + [(1.5, -0.5, 0.0)]
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / np.linalg.norm(g)
    for a, b, c in coeffs:
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(oracle.orthogonalize(g, coeffs, 0.0), (u * s) @ vt, atol=1e-12)


def test_orthogonalize_limits():
    q, _ = np.linalg.qr(np.random.default_rng(0).normal(size=(8, 8)))
    # the cubic iteration keeps an orthogonal matrix's directions and drives the values to 1
    out = oracle.orthogonalize(q, [(1.5, -0.5, 0.0)] * 12, 0.0)
    assert np.allclose(out, q, atol=1e-9)
    assert (oracle.orthogonalize(np.zeros((3, 4)), [(3.0, -4.0, 2.0)], 1e-7) == 0).all()


def test_momentum():
    g, m = np.random.default_rng(0).normal(size=(2, 3, 4))
    buf = torch.tensor(m).lerp(torch.tensor(g), 1 - 0.9)
    new, plain = oracle.momentum_update(g, m, 0.9, False)
    assert np.allclose(new, buf) and np.allclose(plain, buf)
    _, nest = oracle.momentum_update(g, m, 0.9, True)
    assert np.allclose(nest, torch.tensor(g).lerp(buf, 0.9))
