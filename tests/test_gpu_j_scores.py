"""Scores of logits and their gradient against the oracle in 64 bits.

Tolerances.  A probability 2^y, y = c (x - m): three roundings of y (the difference,
c, the product), each 2^-24 |y|, and ex2's 2^-22.  In the sum they are weighted by the
probabilities, whose mean |y| is the entropy at most, ln V / ln 2.  A sum of V values
adds V / 1024 + 32 roundings (two chains a thread of 512, then trees; with fewer
threads the rows are shorter by more).  So s is within
K = 2^-22 + 2^-24 (3 ln V + V / 1024 + 32 + 8) of itself, ln s within K + 2^-24 |ln s|,
and each output adds two roundings of its parts, which are at most its own size, ln V
and the largest |z| in the row.  u / s has K twice, times its size, at most ln V.
Gradients: p carries the rounding of z - lse (2^-24 of max(|z|, |lse|) twice, and that
of lse itself, an input) and ex2's; the factor (G + g_H (d + H)) four roundings of its
parts.  Each output adds half a step of its type."""
import math

import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
import oracle

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
R = 2.0 ** -24


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make(N, V, dtype, seed=0, std=2.5, pitch=None, at=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((N, pitch or V), generator=g) * std
    return x.to(DT[dtype]).cuda()[:, at:at + V]


def make_tokens(N, V, M, seed=1):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, V, (N, M), generator=g, dtype=torch.int32)
    t[torch.rand((N, M), generator=g) < 0.1] = -1
    return t.cuda()


def k_of(V):
    return 4 * R + R * (3 * math.log(V) + V / 1024 + 40)


def near(got, ref, tol):
    got, ref = f64(got), np.asarray(ref)
    fine = np.isfinite(ref)
    assert np.array_equal(fine, np.isfinite(got)) and np.array_equal(np.isnan(ref), np.isnan(got))
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
    off = np.abs(got[fine] - ref[fine])
    assert (off <= np.broadcast_to(tol, ref.shape)[fine]).all(), off.max()


def check_fwd(x, tokens, k, scale, mask, got):
    N, V = x.shape
    lp, ent, lse, top, ids = got
    t2 = None if tokens is None else f64(tokens).astype(int).reshape(N, -1)
    rlp, rent, rlse, rtop, rids = oracle.token_scores(f64(x), t2, k, scale, f64(mask))
    z = np.where(np.isfinite(f64(x)), np.abs(f64(x)) * scale, 0).max(1)
    lnv = math.log(V) + 1
    row = k_of(V) + R * (lnv + 2 * z)
    near(lse, rlse, row + R * np.abs(rlse))
    near(ent, rent, 4 * k_of(V) * lnv + 4 * R * lnv)
    if tokens is not None:
        ref = rlp.reshape(tokens.shape)
        near(lp, ref, (row[:, None] + 3 * R * np.where(np.isfinite(rlp), np.abs(rlp), 0)).reshape(tokens.shape))
    if k:
        near(top, rtop, row[:, None] + 3 * R * np.where(np.isfinite(rtop), np.abs(rtop), 0))
        assert np.array_equal(ids.cpu().numpy(), rids)


# one value, less than a vector, one CTA a row, rows split over clusters of 2, 4 and 8,
# rows too short for that, the vocabularies of the workloads
SHAPES = [(1, 1, 1, 1), (3, 5, 2, 5), (2, 8, 1, 3), (7, 64, 3, 20), (5, 1000, 3, 20), (40, 1003, 1, 64),
          (1, 4097, 128, 64), (2, 32003, 1, 64), (9, 32768, 5, 8), (1, 128256, 1, 20), (33, 9000, 1, 8),
          (70, 20001, 2, 33), (200, 5003, 1, 7), (400, 2050, 1, 12), (3, 152064, 1, 0), (1000, 77, 0, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype):
    N, V, M, k = shape
    x = make(N, V, dtype, N + V)
    tokens = make_tokens(N, V, M) if M else None
    mask = (torch.rand(N, generator=torch.Generator().manual_seed(2)) < 0.8).to(torch.uint8).cuda()
    for scale, mk in ((1.0, None), (0.7, mask)):
        got = eas.token_logprobs_fwd(x, tokens, k, scale, mk)
        assert (got[0] is None) == (M == 0) and (got[3] is None) == (got[4] is None) == (k == 0)
        check_fwd(x, tokens, k, scale, mk, got)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [3, 320])
@pytest.mark.parametrize("V,pitch,at", [(1001, 1013, 3), (4095, 4099, 1), (640, 641, 1), (8192, 8200, 8), (5, 9, 2)])
def test_rows_off_their_vectors(V, pitch, at, N, dtype):
    x = make(N, V, dtype, 5, pitch=pitch, at=at)
    tokens = make_tokens(N, V, 2)
    check_fwd(x, tokens, 5, 1.0, None, eas.token_logprobs_fwd(x, tokens, 5))


def rows_with_ties(V, dtype):
    """Rows whose largest values tie, with few allowed tokens, in order, or with all
    large values in a few of the row's parts."""
    inf = math.inf
    g = torch.Generator().manual_seed(3)
    rows = [torch.zeros(V), torch.full((V,), -3.0), torch.arange(V).float(), -torch.arange(V).float(),
            torch.randint(0, 3, (V,), generator=g).float(), torch.randint(-2, 2, (V,), generator=g) * 0.5]
    for allowed in (1, 2, 17, 90, 600):
        r = torch.full((V,), -inf)
        at = torch.randperm(V, generator=g)[:allowed]
        r[at] = torch.randn(at.numel(), generator=g)
        rows.append(r)
    r = torch.full((V,), -0.0)
    r[1::3] = 0.0
    rows.append(r)
    r = torch.randn(V, generator=g)
    r[torch.randperm(V, generator=g)[:V // 3]] = 4.0
    rows.append(r)
    for vec in (8, 4):
        # large values in 60 of the 512 parts of a slice, whichever the split
        r = torch.randn(V, generator=g)
        part = (torch.arange(V) // vec) % 512
        r = torch.where(part < 60, r.abs() + 10, r)
        rows.append(r)
    r = torch.full((V,), float(torch.finfo(DT[dtype]).min))
    rows.append(r.clone())
    r[:V // 2] = 1.0
    rows.append(r)
    return torch.stack(rows).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("V", [50, 600, 4099, 70000])
def test_ties_and_order(V, many, dtype):
    x = rows_with_ties(V, dtype)
    if many:                                  # enough rows for one CTA each
        x = x.repeat(330 // x.shape[0] + 1, 1)
    x = x.cuda()
    for k in (1, 20, 50):
        got = eas.token_logprobs_fwd(x, None, k)
        n = rows_with_ties(V, dtype).shape[0]
        check_fwd(x[:n], None, k, 1.0, None, [None if t is None else t[:n] for t in got])
        if many:
            # the order of a row's sums goes by its distance from a 16-byte boundary,
            # which the copies do not share; their ids are the same
            for a in range(n, x.shape[0], n):
                assert torch.equal(got[4][:n], got[4][a:a + n])
            check_fwd(x[-n:], None, k, 1.0, None, [None if t is None else t[-n:] for t in got])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [1, 400])
def test_not_finite(N, dtype):
    inf, nan = math.inf, math.nan
    for V in (7, 5000):
        base = make(8, V, dtype, 4)
        base[0, 3], base[1, V - 1], base[2, 0] = nan, inf, -inf
        base[3] = -inf
        base[4, 1], base[4, 2] = nan, inf
        base[5, ::2] = nan
        base[6, 1:] = -inf
        base[7] = nan                            # more NaN than a list of ties takes
        for i in range(8):
            x = base[i:i + 1].repeat(N, 1).contiguous()
            tokens = torch.tensor([[0, 3, V - 1]], dtype=torch.int32, device="cuda").repeat(N, 1)
            got = eas.token_logprobs_fwd(x, tokens, 6)
            check_fwd(x[:1], tokens[:1], 6, 1.0, None, [t[:1] for t in got])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_rows_of_many_kinds(dtype):
    """Rows that take the careful paths among ordinary ones, in the kernel that takes rows
    in turn: each finds the shared memory as the one before left it."""
    V = 30001
    odd = rows_with_ties(V, dtype)
    odd = torch.cat([odd, torch.full((1, V), math.nan, dtype=odd.dtype), torch.full((1, V), -math.inf, dtype=odd.dtype)])
    odd[0, 5] = math.inf
    x = make(700, V, dtype, 8)
    at = torch.arange(0, 700, 9)[:3 * odd.shape[0]]
    x[at] = odd.repeat(3, 1)[:at.numel()].cuda()
    mask = torch.ones(700, dtype=torch.uint8, device="cuda")
    mask[1::3] = 0
    tokens = make_tokens(700, V, 2)
    for k in (3, 64):
        got = eas.token_logprobs_fwd(x, tokens, k, mask=mask)
        pick = torch.cat([at[:2 * odd.shape[0]], torch.arange(1, 700, 40)])
        check_fwd(x[pick], tokens[pick], k, 1.0, mask[pick], [t[pick] for t in got])


@pytest.mark.parametrize("N,V,threads", [(160, 16384, 512), (330, 30000, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_nan_in_nearly_every_threads_part(N, V, threads, dtype):
    """More threads that hold NaN than a list of ties takes, beside some that hold none."""
    x = make(1, V, dtype, 4)
    vec = 8 if dtype == "bf16" else 4
    part = torch.arange(V, device="cuda") // vec % threads
    x[0, part != 5] = math.nan
    x = x.repeat(N, 1)
    tokens = torch.zeros((N, 1), dtype=torch.int32, device="cuda")
    for k in (1, 9, 64):
        got = eas.token_logprobs_fwd(x, tokens, k)
        for i in (0, N - 1):
            check_fwd(x[i:i + 1], tokens[i:i + 1], k, 1.0, None, [t[i:i + 1] for t in got])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [64, 100, 515, 1000, 2047, 5000])
def test_many_alternatives_of_narrow_rows(V, dtype):
    """k close to the number of threads: many candidates for few places, with ties."""
    for N in (3, 400):
        x = make(N, V, dtype, 6)
        x[1] = (x[1] * 2).round() / 2                  # a dozen values
        x[2] = -x[2].abs()
        tokens = make_tokens(N, V, 1)
        for k in (33, 64):
            got = eas.token_logprobs_fwd(x, tokens, k)
            check_fwd(x[:20], tokens[:20], k, 1.0, None, [t[:20] for t in got])


@pytest.mark.parametrize("scale", [2.0 ** -30, 1e-3, 1e3, 2.0 ** 20])
def test_scales(scale):
    for N in (2, 330):
        x = make(N, 30000, "fp32", 3)
        x[0, 7] = -math.inf
        tokens = make_tokens(N, 30000, 2)
        got = eas.token_logprobs_fwd(x, tokens, 9, scale)
        check_fwd(x[:9], tokens[:9], 9, scale, None, [t[:9] for t in got])


def test_inactive_rows_are_not_read():
    x = make(6, 3000, "bf16")
    x[::2] = math.nan
    mask = torch.tensor([0, 1] * 3, dtype=torch.uint8, device="cuda")
    tokens = make_tokens(6, 3000, 2)
    got = eas.token_logprobs_fwd(x, tokens, 4, mask=mask)
    check_fwd(x, tokens, 4, 1.0, mask, got)
    lp, ent, lse, _, _ = got
    g = torch.full((6, 2), math.nan, device="cuda")
    g[1::2] = 1.0
    d = eas.token_logprobs_bwd(g, None, x, tokens, torch.where(mask.bool(), lse, math.nan), ent, mask=mask)
    assert (d[::2] == 0).all() and torch.isfinite(d).all() and (d[1::2] != 0).any()


def test_bad_tokens():
    x = make(3, 100, "fp32")
    tokens = torch.tensor([[5, -1], [7, 100], [9, 3]], dtype=torch.int32, device="cuda")
    ws = torch.full((16,), 255, dtype=torch.uint8, device="cuda")
    lp, ent, lse, _, _ = eas.token_logprobs_fwd(x, tokens, ws=ws)
    assert eas.read_device_status(ws) == 1 and lp[0, 1] == 0 and lp[1, 1] == 0
    g = torch.ones((3, 2), device="cuda")
    d = eas.token_logprobs_bwd(g, None, x, tokens, lse, ent, ws=ws)
    assert eas.read_device_status(ws) == 1
    ref = oracle.token_scores_grad(f64(g), None, f64(x), f64(tokens).astype(int), f64(lse), f64(ent))
    assert np.abs(f64(d) - ref).max() < 1e-5
    tokens[1, 1] = -1
    assert torch.equal(eas.token_logprobs_bwd(g, None, x, tokens, lse, ent, ws=ws), d)
    assert eas.read_device_status(ws) == 0
    tokens[2, 0] = -2
    eas.token_logprobs_fwd(x, tokens, ws=ws)
    assert eas.read_device_status(ws) == 1
    eas.token_logprobs_fwd(x[:0], tokens[:0], 4, ws=ws)
    assert eas.read_device_status(ws) == 0


def check_bwd(x, tokens, g, ge, lse, ent, scale, mask, d, dtype):
    N = x.shape[0]
    t2 = None if tokens is None else f64(tokens).astype(int).reshape(N, -1)
    g2 = None if g is None else f64(g).reshape(N, -1)
    ref = oracle.token_scores_grad(g2, f64(ge), f64(x), t2, f64(lse), f64(ent), scale, f64(mask))
    z = scale * np.where(np.isfinite(f64(x)), f64(x), 0)
    dd = z - f64(lse)[:, None]
    p = np.where(np.isfinite(f64(x)), np.exp(dd), 0)
    ga = np.zeros((N, 1)) if g is None else np.abs(g2 * (t2 >= 0)).sum(1, keepdims=True)
    part = ga + (0 if ge is None else np.abs(f64(ge))[:, None] * (np.abs(dd) + np.abs(f64(ent))[:, None]))
    m = 0 if g is None else t2.shape[1]
    rel = 4 * R + 2 * R * np.abs(dd) + R * (np.abs(z) + np.abs(f64(lse))[:, None])
    tol = scale * p * part * (rel + (8 + m) * R) + HALF[dtype] * np.abs(ref)
    if g is not None:
        hit = np.zeros_like(p)
        for i in range(N):
            for j, t in enumerate(t2[i]):
                if t >= 0:
                    hit[i, t] += abs(g2[i, j])
        tol += scale * hit * (m + 2) * R + HALF[dtype] * scale * 4 * R * hit
    if dtype == "bf16":
        tol += 2.0 ** -133
    else:
        tol += 2.0 ** -125                    # results below the normal range are flushed
    assert (np.abs(f64(d) - ref) <= tol).all(), (np.abs(f64(d) - ref) - tol).max()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dtype):
    N, V, M, _ = shape
    x = make(N, V, dtype, N + V)
    tokens = make_tokens(N, V, M) if M else None
    gen = torch.Generator().manual_seed(9)
    g = torch.randn((N, M), generator=gen).cuda() if M else None
    ge = (torch.randn(N, generator=gen) * 0.1).cuda()
    mask = (torch.rand(N, generator=gen) < 0.8).to(torch.uint8).cuda()
    for scale, mk, h in ((1.0, None, ge), (0.7, mask, ge), (1.0, None, None)):
        _, ent, lse, _, _ = eas.token_logprobs_fwd(x, None, 0, scale, mk)
        d = eas.token_logprobs_bwd(g, h, x, tokens, lse, ent, scale, mk)
        check_bwd(x, tokens, g, h, lse, ent, scale, mk, d, dtype)
        buf = x.clone()
        assert eas.token_logprobs_bwd(g, h, buf, tokens, lse, ent, scale, mk, out=buf) is buf
        assert torch.equal(buf, d)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [2, 700])
def test_backward_pitches_and_repeats(N, dtype):
    V = 1001
    x = make(N, V, dtype, 5, pitch=1013, at=3)
    tokens = torch.randint(0, 4, (N, 9), dtype=torch.int32, device="cuda")      # several times the same
    tokens[:, 4] = V - 1
    tokens[:, 5] = -1
    g = torch.randn((N, 9), device="cuda")
    ge = torch.randn(N, device="cuda")
    _, ent, lse, _, _ = eas.token_logprobs_fwd(x, None, 0)
    d = eas.token_logprobs_bwd(g, ge, x, tokens, lse, ent)
    check_bwd(x, tokens, g, ge, lse, ent, 1.0, None, d, dtype)
    for pitch, at in ((1013, 3), (1016, 5), (1001, 0)):
        wide = torch.full((N, pitch), 7.0, dtype=DT[dtype], device="cuda")
        eas.token_logprobs_bwd(g, ge, x, tokens, lse, ent, out=wide[:, at:at + V])
        assert torch.equal(wide[:, at:at + V], d)
        assert (wide[:, :at] == 7).all() and (wide[:, at + V:] == 7).all()


def test_backward_of_rows_that_allow_few_tokens():
    x = rows_with_ties(4099, "fp32")[6:11].cuda()
    lp, ent, lse, top, ids = eas.token_logprobs_fwd(x, None, 1)
    ge = torch.ones(5, device="cuda")
    g = torch.ones(5, 1, device="cuda")
    d = eas.token_logprobs_bwd(g, ge, x, ids, lse, ent)
    assert (d[x == -math.inf] == 0).all()
    check_bwd(x, ids, g, ge, lse, ent, 1.0, None, d, "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", ["one", "some", "none"])
def test_autograd(shape, dtype):
    N, V, k, scale = 12, 700, 6, 0.8
    x = make(N, V, dtype, 1).contiguous().requires_grad_()
    tokens = {"one": make_tokens(N, V, 1)[:, 0].contiguous(), "some": make_tokens(N, V, 3), "none": None}[shape]
    mask = torch.ones(N, dtype=torch.uint8, device="cuda")
    mask[2] = 0
    lp, ent, top, ids = eas.fused_token_logprobs(x, tokens, k, scale, mask)
    w = torch.randn(N, k, device="cuda")
    loss = (top * w).sum() + 0.3 * ent.sum()
    ref_x = x.detach().double().requires_grad_()
    logp = torch.log_softmax(ref_x * scale, -1)[mask.bool()]
    ref = (logp.gather(1, ids[mask.bool()].long()) * w[mask.bool()]).sum() - 0.3 * (logp.exp() * logp).sum()
    if tokens is not None:
        loss = loss + 2 * lp.sum()
        t = tokens.reshape(N, -1)[mask.bool()].long()
        ref = ref + 2 * torch.where(t >= 0, logp.gather(1, t.clamp(min=0)), 0.0).sum()
    loss.backward()
    ref.backward()
    err = (x.grad.double() - ref_x.grad).abs().max()
    assert err <= HALF[dtype] * ref_x.grad.abs().max() + 1e-5
    # each output alone, and with a broadcast gradient
    for pick in (0, 1, 2):
        y = x.detach().clone().requires_grad_()
        out = eas.fused_token_logprobs(y, tokens, k, scale, mask)[pick]
        if out is not None:
            out.sum().backward()
            assert torch.isfinite(y.grad).all() and (y.grad[2] == 0).all()


def test_empty_and_refusals():
    x = make(4, 50, "fp32")
    t = make_tokens(4, 50, 2)
    out = eas.token_logprobs_fwd(x[:0], t[:0], 3)
    assert out[0].shape == (0, 2) and out[3].shape == (0, 3)
    e = torch.empty(0, device="cuda")
    assert eas.token_logprobs_bwd(e.reshape(0, 2), e, x[:0], t[:0], e, e).shape == (0, 50)
    _, ent, lse, _, _ = eas.token_logprobs_fwd(x)
    g = torch.ones(4, 2, device="cuda")
    for call, err in (
            (lambda: eas.token_logprobs_fwd(x.half()), TypeError),
            (lambda: eas.token_logprobs_fwd(x[0]), ValueError),
            (lambda: eas.token_logprobs_fwd(x.t()), ValueError),
            (lambda: eas.token_logprobs_fwd(x[:1].expand(4, 50)), ValueError),
            (lambda: eas.token_logprobs_fwd(x, t.long()), TypeError),
            (lambda: eas.token_logprobs_fwd(x, t[:3]), ValueError),
            (lambda: eas.token_logprobs_fwd(x, t.cpu()), ValueError),
            (lambda: eas.token_logprobs_fwd(x, t, 51), eas.EasError),
            (lambda: eas.token_logprobs_fwd(make(2, 100, "fp32"), None, 65), eas.EasError),
            (lambda: eas.token_logprobs_fwd(x, t, -1), (eas.EasError, RuntimeError)),
            (lambda: eas.token_logprobs_fwd(x, t, 3, scale=0.0), eas.EasError),
            (lambda: eas.token_logprobs_fwd(x, t, 3, scale=math.nan), eas.EasError),
            (lambda: eas.token_logprobs_fwd(x, torch.zeros(4, 129, dtype=torch.int32, device="cuda")), eas.EasError),
            (lambda: eas.token_logprobs_fwd(x, mask=torch.ones(3, dtype=torch.uint8, device="cuda")), ValueError),
            (lambda: eas.token_logprobs_bwd(g, None, x, None, lse, ent), ValueError),
            (lambda: eas.token_logprobs_bwd(g[:, :1], None, x, t, lse, ent), ValueError),
            (lambda: eas.token_logprobs_bwd(g, None, x, t, lse[:2], ent), ValueError),
            (lambda: eas.token_logprobs_bwd(g, None, x, t, lse, ent, out=x.bfloat16()), TypeError),
            (lambda: eas.token_logprobs_bwd(g, None, x, t, lse, ent, out=x[:, :30]), ValueError),
            (lambda: eas.fused_token_logprobs(x, torch.zeros(4, 120, dtype=torch.int32, device="cuda"), 20), ValueError)):
        with pytest.raises(err):
            call()


def test_writes_stay_inside_their_buffers():
    from test_gpu_9_guard import Guarded
    for N, V, M, k, dtype in ((5, 1003, 3, 7, "bf16"), (400, 1003, 1, 64, "fp32"), (1, 70000, 1, 20, "bf16")):
        gd = Guarded(torch.device("cuda", 0))
        x = gd.view((N, V), DT[dtype])
        x.copy_(make(N, V, dtype, 1))
        t = gd.view((N, M), torch.int32)
        t.copy_(make_tokens(N, V, M))
        f = torch.float32
        out = [gd.view((N, M), f), gd.view((N,), f), gd.view((N,), f), gd.view((N, k), f), gd.view((N, k), torch.int32)]
        got = eas.token_logprobs_fwd(x, t, k, out=out, ws=gd.bytes(16))
        check_fwd(x, t, k, 1.0, None, got)
        d = gd.view((N, V), DT[dtype])
        eas.token_logprobs_bwd(torch.ones_like(out[0]), None, x, t, got[2], got[1], out=d, ws=gd.bytes(16))
        gd.check()


def test_repeats_other_stream_and_graph():
    x, t = make(90, 32003, "bf16"), make_tokens(90, 32003, 2)
    g = torch.randn(90, 2, device="cuda")
    a = eas.token_logprobs_fwd(x, t, 9)
    da = eas.token_logprobs_bwd(g, a[1], x, t, a[2], a[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b = eas.token_logprobs_fwd(x, t, 9)
        db = eas.token_logprobs_bwd(g, b[1], x, t, b[2], b[1])
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = eas.token_logprobs_fwd(x, t, 9)
        dc = eas.token_logprobs_bwd(g, c[1], x, t, c[2], c[1])
    for v in (*c, dc):
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for u, v, w in zip((*a, da), (*b, db), (*c, dc)):
        assert torch.equal(u, v) and torch.equal(u, w)


def test_offsets_beyond_32_bits():
    N, V = 17000, 128256
    x = torch.zeros((N, V), dtype=torch.bfloat16, device="cuda")
    x[-1, 100000], x[-1, 5] = 3.0, 2.0
    t = torch.full((N,), 100000, dtype=torch.int32, device="cuda")
    lp, ent, lse, top, ids = eas.token_logprobs_fwd(x, t, 3)
    ref = math.log(math.exp(3) + math.exp(2) + V - 2)
    assert abs(float(lse[-1]) - ref) < 1e-4 and abs(float(lp[-1]) - 3 + ref) < 1e-4
    assert ids[-1].tolist() == [100000, 5, 0] and ids[-2].tolist() == [0, 1, 2]
    g = torch.ones(N, device="cuda")
    d = eas.token_logprobs_bwd(g, None, x, t, lse, ent, out=x)
    assert abs(float(d[-1, 100000]) - (1 - math.exp(3 - ref))) < 2 ** -8
    assert abs(float(d[-2, 100000]) - 1) < 2 ** -7 and abs(float(d[-1, 5]) + math.exp(2 - ref)) < 2 ** -8 * math.exp(2 - ref) + 1e-7
