"""The differentiable forms in bf16, the type that models are trained in: gradients
come in bf16, the weight's and the table's rounded once from fp32."""
import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
import oracle
from test_gpu_a_norm import EPS, chain, f64, problem, rows

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


@pytest.mark.parametrize("R,H", [(6, 100), (130, 4096), (37, 1003)])
@pytest.mark.parametrize("residual,mask", [(True, "some"), (False, None)])
def test_rmsnorm(R, H, residual, mask):
    x, w, r, m = problem(R, H, "bf16", residual, mask, seed=R)
    leaves = [t.requires_grad_() for t in (x, w, r) if t is not None]
    y, s, _, _ = eas.fused_rmsnorm(x, w, r, EPS, m)
    gy, gs = rows((R, H), "bf16", 7, 0.1), rows((R, H), "bf16", 8, 0.1)
    outs, grads = ((y, s), (gy, gs)) if residual else ((y,), (gy,))
    got = torch.autograd.grad(outs, leaves, grads)
    S, D, W = f64((s if residual else x).detach()), f64(gy), f64(w.detach())
    add = f64(gs) if residual else None
    rdx, rdw = oracle.rmsnorm_grad(D, S, W, EPS, add, None if m is None else f64(m))
    on = np.ones((R, 1)) if m is None else f64(m)[:, None]
    rstd = 1 / np.sqrt((S * S).mean(1, keepdims=True) + EPS)
    g, n = np.abs(D * W), np.abs(S) * rstd
    terms = rstd * (g + n * (g * n).mean(1, keepdims=True)) * on
    tol = HALF * np.abs(rdx) + (2.5 * chain(H) + 12) * 2.0 ** -24 * terms + 2.0 ** -23 * (0 if add is None else np.abs(add))
    assert all(t.dtype == torch.bfloat16 for t in got)
    assert (np.abs(f64(got[0]) - rdx) <= tol).all()
    # fp32 sums over at most R rows, then bf16
    k = (min(R, 64) + R / 64 + chain(H) / 2 + 16) * 2.0 ** -24
    assert (np.abs(f64(got[1]) - rdw) <= HALF * np.abs(rdw) + 2 * k * (np.abs(D) * n * on).sum(0)).all()
    if residual:
        assert torch.equal(got[2], got[0])


@pytest.mark.parametrize("T,H,V", [(50, 100, 30), (700, 1003, 90), (5000, 64, 777)])
def test_embedding(T, H, V):
    from test_gpu_b_embed import make_ids
    table = rows((V, H), "bf16", 0).requires_grad_()
    ids = make_ids(T, V, "padded")
    out = eas.fused_embedding(torch.from_numpy(ids).cuda(), table, 3.0)
    g = rows((T, H), "bf16", 1)
    out.backward(g)
    assert out.dtype == table.grad.dtype == torch.bfloat16
    ref, absum = oracle.embed_grad(ids, f64(g), V, 3.0), oracle.embed_grad(ids, np.abs(f64(g)), V, 3.0)
    n = np.bincount(ids[ids >= 0], minlength=V)[:, None]
    assert (np.abs(f64(table.grad) - ref) <= HALF * np.abs(ref) + 2 * (n + 1) * 2.0 ** -24 * absum).all()
