"""Scores of logits far from 0: masked ones at -1e30 or the like among others or alone,
large ones, and scales that make them large.  The order of a row's values must not matter.

Tolerances as for other logits, but relative to what a row's likely values differ by: from
2^26 on differences are taken before they are scaled, which rounds twice, and c once; below
that the rounding of the largest z counts twice."""
import math

import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
import oracle
from test_gpu_j_scores import R, DT, f64, k_of, make, make_tokens, near

pytestmark = pytest.mark.gpu


def check(x, tokens, k, scale, got):
    x = f64(x)
    N, V = x.shape
    t = f64(tokens).astype(int)
    scale = float(np.float32(scale))
    rlp, rent, rlse, rtop, rids = oracle.token_scores(x, t, k, scale)
    z = scale * x
    likely = z >= z.max(1, keepdims=True) - 200
    far = np.abs(z).max(1, where=likely, initial=0)
    far = np.where(far >= 2.0 ** 25, 0, far)
    lnv = math.log(V) + 1
    row = k_of(V) + R * (lnv + 2 * far)
    lp, ent, lse, top, ids = got
    near(lse, rlse, row + 3 * R * np.abs(rlse))
    near(ent, rent, 4 * k_of(V) * lnv + 4 * R * lnv)
    near(lp, rlp, row[:, None] + 4 * R * np.where(np.isfinite(rlp), np.abs(rlp), 0))
    near(top, rtop, row[:, None] + 4 * R * np.where(np.isfinite(rtop), np.abs(rtop), 0))
    assert np.array_equal(ids.cpu().numpy(), rids)


def rows(V, dtype, value):
    """All at `value`; all but a few; a few; the first half; the second half."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn((6, V), generator=g)
    for i, share in enumerate((1.0, 0.999, 0.5, 0.01)):
        x[i][torch.rand(V, generator=g) < share] = value
    x[1, V // 3] = 0.5
    x[4, :V // 2] = value
    x[5, V // 2:] = value
    return x.to(DT[dtype])


# one CTA a row, a cluster a row, rows in turn by groups of four and of eight vectors
KERNELS = [(6, 1000), (400, 900), (6, 30001), (330, 16401), (330, 40003)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [-1e8, -3e9, -1e10, -1e15, -1e30, -1e38, 1e10, 1e30])
@pytest.mark.parametrize("N,V", KERNELS)
def test_masked_by_a_large_number(N, V, value, dtype):
    x = rows(V, dtype, value)
    x = x.repeat((N + 5) // 6, 1)[:N].cuda()
    tokens = make_tokens(N, V, 3)
    got = eas.token_logprobs_fwd(x, tokens, 7)
    check(x[:6], tokens[:6], 7, 1.0, [v[:6] for v in got])
    check(x[-6:], tokens[-6:], 7, 1.0, [v[-6:] for v in got])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("level", [2.0 ** 20, 1.1 * 2.0 ** 25, 2.0 ** 26 / 1.4426951, 2.0 ** 26, 2.0 ** 31, 1e25, 1e37])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("N,V", KERNELS)
def test_rows_at_a_large_number(N, V, sign, level, dtype):
    """Every value within a few of the type's steps of `level`, times a scale that leaves a
    few units between them."""
    eps = torch.finfo(DT[dtype]).eps
    g = torch.Generator().manual_seed(2)
    x = (sign * level * (1 + eps * torch.randint(-3, 4, (min(N, 12), V), generator=g, dtype=torch.float64))).to(DT[dtype])
    x = x.repeat(N // x.shape[0] + 1, 1)[:N].cuda()
    tokens = make_tokens(N, V, 3)
    for scale in (1.0, 0.7):
        got = eas.token_logprobs_fwd(x, tokens, 7, scale)
        check(x[:6], tokens[:6], 7, scale, [v[:6] for v in got])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [2.0 ** 22, 2.0 ** 25, 1e8, 2.0 ** 40])
@pytest.mark.parametrize("N,V", KERNELS)
def test_large_scales(N, V, scale, dtype):
    x = make(N, V, dtype, 3)
    x[1] = -x[1].abs() - 1
    tokens = make_tokens(N, V, 2)
    got = eas.token_logprobs_fwd(x, tokens, 7, scale)
    check(x[:6], tokens[:6], 7, scale, [v[:6] for v in got])
