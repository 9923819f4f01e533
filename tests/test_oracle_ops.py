"""Pins of the oracle's operators around the LM head (CPU only): gradients
against central differences, closed forms, masks, and planted mistakes."""
import numpy as np
import pytest

import oracle


def fd(f, x, h=1e-6):
    """Central differences of the scalar f() in the entries of x, in place."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        a = f()
        x[i] = keep - h
        b = f()
        x[i] = keep
        g[i] = (a - b) / (2 * h)
    return g


@pytest.mark.parametrize("mask", [None, [1, 0, 1, 1], [0, 0, 0, 0]])
def test_rmsnorm_gradient_is_the_derivative(mask):
    rng = np.random.default_rng(1)
    x, r, w = rng.standard_normal((4, 6)), rng.standard_normal((4, 6)), rng.standard_normal(6)
    gy, gs = rng.standard_normal((4, 6)), rng.standard_normal((4, 6))

    def loss():
        y, s = oracle.rmsnorm(x, w, 1e-3, r, mask)
        return (gy * y).sum() + (gs * s).sum()

    _, s = oracle.rmsnorm(x, w, 1e-3, r, mask)
    dx, dw = oracle.rmsnorm_grad(gy, s, w, 1e-3, gs, mask)
    # central differences are off by h^2 f'''/6 and by the rounding of f over h
    for arr, want in ((x, dx), (r, dx), (w, dw)):
        np.testing.assert_allclose(fd(loss, arr), want, rtol=1e-6, atol=1e-8)


def test_rmsnorm_closed_forms():
    y, s = oracle.rmsnorm(np.full((1, 8), -3.0), np.full(8, 2.0), 1e-300)
    np.testing.assert_allclose(y, -2.0, rtol=1e-15)
    y, _ = oracle.rmsnorm(np.zeros((1, 8)), np.ones(8), 1e-6)
    assert (y == 0).all()
    y, s = oracle.rmsnorm(np.array([[np.nan, 1.0], [3.0, 4.0]]), np.ones(2), 1e-6, mask=[0, 1])
    assert (y[0] == 0).all() and np.isfinite(y[1]).all()


def test_rmsnorm_difference_rejects_a_dropped_mean():
    rng = np.random.default_rng(2)
    x, w, gy = rng.standard_normal((2, 5)), rng.standard_normal(5), rng.standard_normal((2, 5))
    want = fd(lambda: (gy * oracle.rmsnorm(x, w, 1e-3)[0]).sum(), x)
    rms = np.sqrt((x * x).mean(1, keepdims=True) + 1e-3)
    assert not np.allclose(gy * w / rms, want, rtol=1e-3, atol=1e-6)


def test_embedding_gradient_is_the_derivative():
    rng = np.random.default_rng(3)
    ids = np.array([2, -1, 0, 2, 9, 2])
    table, g = rng.standard_normal((4, 3)), rng.standard_normal((6, 3))
    dw = oracle.embed_grad(ids, g, 4, 1.5)
    np.testing.assert_allclose(fd(lambda: (g * oracle.embed(ids, table, 1.5)).sum(), table), dw,
                               rtol=1e-6, atol=1e-8)
    assert (oracle.embed(ids, table, 1.5)[[1, 4]] == 0).all()     # padding and a bad id
    assert (dw[[1, 3]] == 0).all()


def test_clip_closed_forms():
    g = [np.array([3.0]), np.array([0.0, 4.0])]
    norm, out = oracle.clip_grads(g, 1.0)
    assert norm == 5.0
    np.testing.assert_allclose(np.concatenate(out), np.array([3.0, 0, 4.0]) / (5 + 1e-6), rtol=1e-15)
    _, out = oracle.clip_grads(g, 10.0)
    np.testing.assert_array_equal(np.concatenate(out), [3.0, 0, 4.0])
    norm, out = oracle.clip_grads([np.array([np.inf, 1.0])], 1.0)
    assert np.isinf(norm) and out[0][1] == 1.0
