"""The RMS norm with an eps far below 1e-30 against the oracle in 64 bits.

Tolerances: 64 terms a thread and ten levels of a tree give a row statistic 74 roundings,
of which rstd takes half, with eight more operations; one rounding to fp32."""
import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
import oracle

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("eps", [2e-38, 1e-33])
@pytest.mark.parametrize("H", [96, 1000])
def test_forward_and_backward(H, eps):
    g = torch.Generator().manual_seed(H)
    x, dy = torch.randn((7, H), generator=g).cuda(), torch.randn((7, H), generator=g).cuda()
    w = (1 + 0.3 * torch.randn(H, generator=g)).cuda()
    tol = 50 * 2.0 ** -24
    y, _, _, _ = eas.rmsnorm_fwd(x, w, eps)
    ry, _ = oracle.rmsnorm(f64(x), f64(w), eps)
    assert (np.abs(f64(y) - ry) <= tol * np.abs(ry)).all()
    dx, dw = eas.rmsnorm_bwd(dy, x, w, eps)
    rdx, rdw = oracle.rmsnorm_grad(f64(dy), f64(x), f64(w), eps)
    for a, r in ((dx, rdx), (dw, rdw)):
        assert np.linalg.norm(f64(a) - r) <= 2 * tol * np.linalg.norm(r)
    zero = torch.zeros(2, H, device="cuda")
    assert (eas.rmsnorm_fwd(zero, w, eps)[0] == 0).all()
