"""The gradient at rows whose logits lie far from 0: a probability is 1 at most, however
much of z - lse is the rounding of lse."""
import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
from test_gpu_j_scores import DT, check_bwd, f64, make_tokens

pytestmark = pytest.mark.gpu


def rows(V, value, dtype):
    """All masked by `value`, with steps of its type between them; all but one; half."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn((3, V), generator=g)
    eps = torch.finfo(DT[dtype]).eps
    x[0] = value * (1 + eps * torch.randint(-2, 3, (V,), generator=g))
    x[1] = value
    x[1, V // 3] = 0.5
    x[2, torch.rand(V, generator=g) < 0.5] = value
    return x.to(DT[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [-1e6, -1e9, -1e10, -1e30, -3e38, 1e9, 1e30])
@pytest.mark.parametrize("V", [1003, 30001])
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_masked_by_a_large_number(V, scale, value, dtype):
    x = rows(V, value, dtype)
    t = make_tokens(3, V, 2)
    _, ent, lse, _, _ = eas.token_logprobs_fwd(x, None, 0, scale)
    g, ge = torch.ones(3, 2, device="cuda"), torch.full((3,), 0.1, device="cuda")
    d = eas.token_logprobs_bwd(g, ge, x, t, lse, ent, scale)
    # G and g_H (z - lse + H) times a p of 1 at most, and each token's own gradient
    most = scale * (2 + 0.1 * (1 + f64(ent)) + 2)[:, None] * (1 + 2.0 ** -7)
    assert (np.abs(f64(d)) <= most).all()
    if value < 0:                             # with an lse near 0: what the formula says
        check_bwd(x[1:], t[1:], g[1:], ge[1:], lse[1:], ent[1:], scale, None, d[1:], dtype)
    none = torch.zeros(3, 2, device="cuda"), torch.zeros(3, device="cuda")
    assert (eas.token_logprobs_bwd(*none, x, t, lse, ent, scale) == 0).all()


def test_a_row_with_nan_keeps_it():
    x = torch.zeros(2, 40, device="cuda")
    x[1, 3] = float("nan")
    t = torch.zeros(2, dtype=torch.int32, device="cuda")
    _, ent, lse, _, _ = eas.token_logprobs_fwd(x, t)
    d = eas.token_logprobs_bwd(torch.ones(2, device="cuda"), None, x, t, lse, ent)
    assert torch.isfinite(d[0]).all() and torch.isnan(d[1]).all()
