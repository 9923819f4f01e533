"""Values of the operators around the LM head to the last rounding.

The inputs make every step but the ones under test exact, so the tolerance is the
count of the roundings that the definition needs, half a step each."""
import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas

pytestmark = pytest.mark.gpu

U = 2.0 ** -24          # half a step of fp32


@pytest.mark.parametrize("into", ["place", "fp32"])
def test_clipping_factor(into):
    """Integers, so the sum of squares is exact: the factor is rounded to fp32 once
    and each product once more."""
    rng = np.random.default_rng(3)
    for i in range(40):
        g = [rng.integers(-9, 10, 500 + i), rng.integers(-9, 10, 77)]
        t = [torch.from_numpy(g[0].astype(np.float32)).cuda(), torch.from_numpy(g[1].astype(np.float32)).cuda()]
        max_norm = float(np.float32(rng.uniform(0.1, 20.0)))
        norm64 = np.sqrt(float((g[0] ** 2).sum() + (g[1] ** 2).sum()))
        c = max_norm / (norm64 + 1e-6)
        assert c < 1
        out = t if into == "place" else [torch.empty_like(x) for x in t]
        norm = eas.clip_grad_norm(t, max_norm, out=None if into == "place" else out)
        assert abs(float(norm) - norm64) <= U * norm64
        for x, o in zip(g, out):
            ref = x * c
            assert (np.abs(o.double().cpu().numpy() - ref) <= (2 * U + 2.0 ** -40) * np.abs(ref)).all()
