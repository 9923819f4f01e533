"""The log-sum-exp of rows that lie off 0, from which the gradient takes its
probabilities: within its own rounding, 2^-24 of it, and what the sums of the differences
leave (their K, and two roundings of ln V)."""
import math

import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
import oracle
from test_gpu_j_scores import R, f64, k_of, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", [30.0, -1e3, 1e4, 1e6])
@pytest.mark.parametrize("scale", [1.0, 0.7])
@pytest.mark.parametrize("N,V", [(200, 1000), (40, 20001), (330, 16401)])
def test_lse_to_its_last_step(N, V, scale, at):
    x = make(N, V, "fp32", 1) + at + 0.37 * torch.arange(N, device="cuda")[:, None]
    _, _, lse, _, _ = eas.token_logprobs_fwd(x, None, 0, scale)
    pick = slice(0, 40)
    ref = oracle.token_scores(f64(x[pick]), scale=float(np.float32(scale)))[2]
    tol = R * np.abs(ref) + k_of(V) + 2 * R * (math.log(V) + 1)
    assert (np.abs(f64(lse[pick]) - ref) <= tol).all(), (np.abs(f64(lse[pick]) - ref) / tol).max()
