"""What the orthogonalised update keeps of a gradient without full rank, in each of its
kernels, and over more than five steps.

Tolerances, of the update's 2-norm.  Its rounding to bf16: a step of 2^-7 over sqrt(12),
over values spread evenly in their logarithm, 1.66e-3.  A rounding to fp16 is an eighth of
that.  In a step that takes a singular value s to p(s) = a s + b s^3 + c s^5, A is rounded
(for b A, and twice for c A A), X for its product with B - a, and B: each relative to its
term, |b| s^2, |c| s^4 twice, |b s^2 + c s^4| and p(s) / s, with X of size s beside the
result of size p(s).  All of these add up in squares; a quarter more is allowed for those
that do not average out.  The products' fp32 sums leave 2^-23 of X for every 16 terms of
theirs, in squares again, and what of it lies in directions that the gradient does not have
grows by a in each step.  X's own rounding, to 22 bits, is below that."""
import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
import oracle

pytestmark = pytest.mark.gpu

ABC = eas.NEWTON_SCHULZ


def tolerance(x, coeffs):
    n = min(x.shape)
    gram = x @ x.T if x.shape[0] == n else x.T @ x
    q = np.maximum(np.linalg.eigvalsh(gram), 0.0)
    q /= q.sum()
    off, half = 1.66e-3 ** 2, 1.66e-3 / 8
    for a, b, c in coeffs:
        u, v = b * q, c * q * q
        p = a + u + v
        off += half ** 2 * (q * (u * u + 2 * v * v + (u + v) ** 2 + p * p)).sum() / (q * p * p).sum()
        q = q * p * p
    growth = np.prod([abs(c[0]) for c in coeffs])
    return 1.25 * np.sqrt(off) + growth * 2.0 ** -23 * np.sqrt(n / 16 + 1)


def of_rank(shape, r, seed):
    L, n, m = shape
    g = torch.Generator().manual_seed(seed)
    return torch.randn((L, n, r), generator=g) @ torch.randn((L, r, m), generator=g)


def check(g, coeffs=(ABC,) * 5):
    g = g.cuda()
    out = eas.orthogonalize(g, len(coeffs), list(coeffs))
    L = g.shape[0]
    for i in {0, L // 2, L - 1}:
        x = g[i].double().cpu().numpy()
        ref, tol = oracle.orthogonalize(x, coeffs, 1e-7), tolerance(x, coeffs)
        off = np.linalg.norm(out[i].double().cpu().numpy() - ref) / np.linalg.norm(ref)
        assert off <= tol, (i, off, tol)


# one CTA a matrix (up to six, seven and eight blocks of columns); half tiles; X X^T in
# parts; whole tiles; pairs of SMs
SHAPES = [(2, 128, 128), (2, 300, 100), (3, 128, 384), (3, 100, 448), (200, 65, 500), (2, 512, 128), (1, 128, 513),
          (1, 256, 512), (1, 513, 257), (1, 200, 3001), (1, 3001, 200), (30, 256, 512), (1, 1200, 1100),
          (16, 520, 1100), (12, 1100, 640)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("rank", [1, 2, 8, 40])
def test_low_rank(shape, rank):
    check(of_rank(shape, rank, rank))


@pytest.mark.parametrize("shape", SHAPES)
def test_ill_conditioned(shape):
    L, n, m = shape
    r = min(n, m)
    g = torch.Generator().manual_seed(7)
    u, v = (torch.linalg.qr(torch.randn((k, r), generator=g, dtype=torch.float64))[0] for k in (n, m))
    x = ((u * torch.logspace(0, -4, r, dtype=torch.float64)) @ v.T).float()
    check(x.expand(L, n, m).contiguous())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(2, 128, 128), (2, 128, 500), (1, 256, 512), (1, 200, 3001), (30, 256, 512), (16, 520, 1100)])
@pytest.mark.parametrize("steps", [6, 7, 8])
@pytest.mark.parametrize("rank", [1, 8])
def test_more_steps(shape, steps, rank, dtype):
    check(of_rank(shape, rank, steps).to(dtype), (ABC,) * steps)


@pytest.mark.parametrize("shape", [(2, 128, 128), (1, 256, 512), (30, 256, 512), (16, 520, 1100)])
@pytest.mark.parametrize("rank", [1, 8])
def test_a_triple_for_each_step(shape, rank):
    """The first ones steep; singular values stay below 2."""
    each = [(7.0, -18.0, 12.5), (4.0, -2.9, 0.55), (3.8, -2.8, 0.54), (3.2, -2.4, 0.48), (2.2, -1.6, 0.4), (1.7, -1.1, 0.35)]
    check(of_rank(shape, rank, 5), each)


@pytest.mark.parametrize("n,m", [(1, 2), (2, 2), (2, 16), (3, 5), (5, 3), (4, 4), (8, 8), (64, 8), (16, 30), (31, 33)])
@pytest.mark.parametrize("rank", [1, 2, 64])
def test_few_rows(n, m, rank):
    """Single singular values: what the roundings of a step leave, about 1e-3 of one (four of
    2^-12 on terms of a few times the result), the next step can carry 1.7 times further (the
    most that p' is up to the largest p, 1.13): 1e-3 (1 + 1.7 + ... + 1.7^4) = 1.9e-2, and
    the output's rounding."""
    g = of_rank((2000, n, m), rank, 3).cuda()
    out = eas.orthogonalize(g).double()
    x = g.double()
    x = x / (x.flatten(1).norm(dim=1)[:, None, None] + 1e-7)
    for a, b, c in (ABC,) * 5:
        q = x @ x.mT
        x = a * x + (b * q + c * q @ q) @ x
    off = (out - x).flatten(1).norm(dim=1) / x.flatten(1).norm(dim=1)
    assert float(off.max()) <= 2.1e-2 and float(off.mean()) <= 5e-3


@pytest.mark.parametrize("shape", [(3, 100, 500), (2, 449, 128), (5, 128, 385), (4, 60, 384), (2, 128, 512)])
def test_workspace_of_small_matrices(shape):
    """lo beyond shared memory: inside its workspace, whatever that held, and the same again."""
    from test_gpu_9_guard import Guarded
    gd = Guarded(torch.device("cuda", 0))
    g = of_rank(shape, 8, 1).cuda()
    ws = gd.bytes(eas.orthogonalize_workspace_size(*shape))
    ws.fill_(0xff)
    out = gd.view(shape, torch.bfloat16)
    eas.orthogonalize(g, ws=ws, out=out)
    assert eas.read_device_status(ws) == 0 and torch.equal(out, eas.orthogonalize(g))
    gd.check()
