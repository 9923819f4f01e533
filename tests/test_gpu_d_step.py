"""The operators together: the example's training step against float64 autograd
on the host, and its loss going down."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

# Every tensor between two operators is rounded to bf16 (2^-8 of it) about six
# times on the way from the loss to the table's gradient, and the rounding errors
# are independent: about sqrt(6) 2^-8 = 1 % of the gradient's norm.  e4m3 logits
# move the probabilities by their own 2^-4 a product, averaged over H products.
FRO = {False: 0.02, True: 0.1}


def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("fp8", [False, True])
def test_gradients_match_float64_autograd(fp8):
    import tied_step as ex
    T, V, H, beta = 700, 900, 256, 0.01
    m, b = ex.make_model(V, H, 3), ex.make_batch(T, V, 4)
    _, got = ex.gradients(m, b, beta, fp8)
    table, layer, gain = (t.double().cpu().requires_grad_() for t in (m.table, m.layer, m.gain))
    ids, on = b["ids"].cpu().long(), b["mask"].cpu().bool()
    x = torch.where((ids >= 0)[:, None], table[ids.clamp(min=0)], torch.zeros(())) * m.scale
    s = x + torch.tanh(x @ layer)
    y = s / (s.square().mean(-1, keepdim=True) + ex.EPS).sqrt() * gain
    logp = torch.log_softmax(y @ table.t(), -1)
    lp = logp.gather(1, b["targets"].cpu().long()[:, None])[:, 0]
    ent = -(logp.exp() * logp).sum(-1)
    (-(b["advantage"].cpu().double() * lp + beta * ent)[on].sum()).backward()
    for k, ref in (("table", table.grad), ("layer", layer.grad), ("gain", gain.grad)):
        assert rel(got[k], ref) <= FRO[fp8], k


@pytest.mark.parametrize("fp8", [False, True])
def test_steps_lower_the_loss(fp8):
    import tied_step as ex
    m, b = ex.make_model(600, 256), ex.make_batch(512, 600)
    b["advantage"] = b["advantage"].abs()
    losses, norms = zip(*(ex.step(m, b, fp8=fp8) for _ in range(8)))
    assert losses[-1] < losses[0] and all(torch.isfinite(n).all() for n in norms)
