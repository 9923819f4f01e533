"""The RMS norm and its backward against the oracle in 64 bits.

Tolerances.  A row statistic is a sum of at most n = 64 terms a thread and ten
levels of a tree (long rows: H / 1024 terms and the tree), so its relative
error is at most about (n + 10) 2^-24 of the sum of the absolute terms; rstd
takes half of that and two steps of rsqrt.  Each output is then a handful of
fp32 operations and one rounding to its type, half a step: 2^-8 relative for
bf16, 2^-24 for fp32, 2^-4 for e4m3 (2^-10 absolute below its normal range)."""
import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
import oracle
from entropy_active_span_gb300 import workloads as W

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def chain(H):
    """Roundings of a row statistic."""
    return 64 + 10 if H <= 8192 else max(64, H / 1024) + 10


def f64(t):
    return t.double().cpu().numpy()


def rows(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).cuda()


def problem(R, H, dtype, residual, mask, seed=0):
    x = rows((R, H), dtype, seed)
    w = (1 + rows((H,), "fp32", seed + 1, 0.3)).to(DT[dtype])
    r = rows((R, H), dtype, seed + 2, 2.0) if residual else None
    m = None
    if mask == "some":
        m = (torch.rand(R, generator=torch.Generator().manual_seed(seed + 3)) < 0.6).to(torch.uint8)
        m[:1], m[R - 1:] = 0, 1
        m = m.cuda()
    elif mask == "empty":
        m = torch.zeros(R, dtype=torch.uint8, device="cuda")
    return x, w, r, m


def check_fwd(x, w, r, m, y, q, scale, s):
    H = x.shape[1]
    ry, rs = oracle.rmsnorm(f64(x), f64(w), EPS, None if r is None else f64(r),
                            None if m is None else f64(m))
    k = (chain(H) / 2 + 8) * 2.0 ** -24
    half = HALF[x.dtype]
    if r is not None:
        assert (np.abs(f64(s) - rs) <= (half + 2.0 ** -24) * np.abs(rs)).all()
    # cancellation in x + r happens before the norm: its rounding, 2^-24 of the
    # sum, scales with |s| itself
    tol = (half + k + 2.0 ** -24) * np.abs(ry)
    if y is not None:
        assert (np.abs(f64(y) - ry) <= tol).all()
    if q is not None:
        amax = np.abs(ry).max(axis=1)
        sc = np.where(amax == 0, 1.0, amax / 448)
        assert (np.abs(f64(scale) - sc) <= (k + 2.0 ** -23) * sc).all()
        val = oracle.e4m3_decode(q.cpu().numpy()) * f64(scale)[:, None]
        # half an e4m3 step of the value, and the rounding of y, 448 / amax and the product
        assert (np.abs(val - ry) <= np.maximum(2.0 ** -4 * np.abs(ry), 2.0 ** -10 * sc[:, None])
                + 4 * k * np.abs(ry) + 2.0 ** -22 * np.abs(ry)).all()


SHAPES = [(1, 1), (3, 7), (1, 128), (5, 128), (2, 320), (37, 1003), (9, 1088), (130, 4096),
          (3, 8192), (2, 8191), (3, 16384), (2, 32768), (2, 32776), (1, 40001),
          (1300, 100), (1300, 101), (700, 2047), (650, 2052), (320, 8189), (20000, 33), (9000, 128),
          (900, 150), (700, 333), (1100, 601), (800, 192)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,H", SHAPES)
def test_forward(R, H, dtype):
    for residual, mask, e4m3 in ((True, "some", True), (False, None, False), (False, "some", True)):
        x, w, r, m = problem(R, H, dtype, residual, mask, seed=R * H)
        y, q, scale, s = eas.rmsnorm_fwd(x, w, EPS, r, m, want_e4m3=e4m3)
        if not residual:
            assert s is x
        check_fwd(x, w, r, m, y, q, scale, s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,H", SHAPES + [(700, 256), (2500, 64)])
def test_backward(R, H, dtype):
    for ds, mask in ((True, "some"), (False, None), (False, "some")):
        s, w, d, m = problem(R, H, dtype, ds, mask, seed=R + H)
        dy = rows((R, H), dtype, R + 5, 0.1)
        dx, dw = eas.rmsnorm_bwd(dy, s, w, EPS, d, m)
        S, D, Wt = f64(s), f64(dy), f64(w)
        rdx, rdw = oracle.rmsnorm_grad(D, S, Wt, EPS, None if d is None else f64(d),
                                       None if m is None else f64(m))
        on = np.ones((R, 1)) if m is None else f64(m)[:, None]
        rstd = 1 / np.sqrt((S * S).mean(1, keepdims=True) + EPS)
        g, n = np.abs(D * Wt), np.abs(S) * rstd
        # the terms of dx in absolute values, each with the error of the two sums
        terms = rstd * (g + n * (g * n).mean(1, keepdims=True)) * on
        k = (2.5 * chain(H) + 12) * 2.0 ** -24
        tol = HALF[s.dtype] * np.abs(rdx) + k * terms + 2.0 ** -23 * (0 if d is None else np.abs(f64(d)))
        assert (np.abs(f64(dx) - rdx) <= tol).all()
        # a sum of at most R rounded products
        tol = (min(R, 64) + R / 64 + chain(H) / 2 + 16) * 2.0 ** -24 * (np.abs(D) * n * on).sum(0)
        assert (np.abs(f64(dw) - rdw) <= tol + 1e-300).all()
        again = eas.rmsnorm_bwd(dy, s, w, EPS, d, m)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_codes_are_the_quantiser_s():
    """In fp32 y is stored unrounded, so quantising it must give the same codes."""
    x, w, r, _ = problem(40, 1024, "fp32", True, None, seed=4)
    y, q, scale, _ = eas.rmsnorm_fwd(x, w, EPS, r, want_e4m3=True)
    q2, scale2 = eas.quantize_rows_e4m3(y)
    assert torch.equal(q, q2) and torch.equal(scale, scale2)


@pytest.mark.parametrize("H", [128, 1003, 4096, 40001])
def test_inactive_rows_are_not_looked_at(H):
    """NaN, infinities and the type's lowest value in inactive rows stay there."""
    for dtype in ("bf16", "fp32"):
        x, w, _, _ = problem(6, H, dtype, False, None, seed=H)
        low = torch.finfo(DT[dtype]).min
        x[0], x[2], x[4] = float("nan"), float("inf"), low
        m = torch.tensor([0, 1, 0, 1, 0, 1], dtype=torch.uint8, device="cuda")
        y, q, scale, _ = eas.rmsnorm_fwd(x, w, EPS, mask=m, want_e4m3=True)
        assert (y[::2] == 0).all() and (q[::2] == 0).all() and (scale[::2] == 1).all()
        assert torch.isfinite(y).all() and (y[1::2] != 0).any()
        dy = x.clone()
        dx, dw = eas.rmsnorm_bwd(dy, x, w, EPS, mask=m)
        assert (dx[::2] == 0).all() and torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("H", [64, 1003, 40001])
def test_empty_mask_and_no_rows(H):
    x, w, r, m = problem(5, H, "bf16", True, "empty", seed=H)
    y, q, scale, s = eas.rmsnorm_fwd(x, w, EPS, r, m, want_e4m3=True)
    assert (y == 0).all() and (q == 0).all() and (scale == 1).all()
    assert torch.equal(s, (x.float() + r.float()).bfloat16())       # the residual stream goes on
    dx, dw = eas.rmsnorm_bwd(x, s, w, EPS, ds=r, mask=m)
    assert torch.equal(dx, r) and (dw == 0).all()
    none = x[:0]
    y, q, scale, s = eas.rmsnorm_fwd(none, w, EPS, none, want_e4m3=True)
    assert y.shape == (0, H) and scale.numel() == 0
    dx, dw = eas.rmsnorm_bwd(none, none, w, EPS)
    assert dx.shape == (0, H) and (dw == 0).all()


def test_zero_and_tiny_rows():
    x = torch.zeros(3, 256, device="cuda")
    x[1, 5], x[2] = 1e-30, 1e-12
    w = torch.full((256,), 1e-20, device="cuda")
    y, q, scale, _ = eas.rmsnorm_fwd(x, w, EPS, want_e4m3=True)
    assert torch.isfinite(y).all() and torch.isfinite(scale).all()
    assert (q[:2] == 0).all() and (scale[:2] == 1).all()       # amax 0, and 1e-47 flushed
    # row 2: y = 1e-12 / 1e-3 * 1e-20 = 1e-29, all equal: code 448
    assert (oracle.e4m3_decode(q[2].cpu().numpy()) == 448).all()


def test_nan_in_an_active_row_shows():
    x, w, _, _ = problem(2, 128, "fp32", False, None)
    x[0, 3] = float("nan")
    y, q, _, _ = eas.rmsnorm_fwd(x, w, EPS, want_e4m3=True)
    assert torch.isnan(y[0]).all() and torch.isfinite(y[1]).all()
    assert ((q[0] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("H", [256, 1003, 40001])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_sum_in_place(H, into):
    x, w, r, m = problem(7, H, "bf16", True, "some", seed=9)
    want = eas.rmsnorm_fwd(x, w, EPS, r, m, want_e4m3=True)
    buf = x if into == "x" else r
    got = eas.rmsnorm_fwd(x, w, EPS, r, m, want_e4m3=True, out=(None, None, None, buf))
    assert got[3].data_ptr() == buf.data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    ds = rows((7, H), "bf16", 3)
    dy = rows((7, H), "bf16", 4)
    a = eas.rmsnorm_bwd(dy, want[3], w, EPS, ds.clone(), m)
    b = eas.rmsnorm_bwd(dy, want[3], w, EPS, ds, m, dx=ds)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_outputs_are_optional():
    x, w, r, _ = problem(5, 512, "bf16", True, None)
    y, q, scale, s = eas.rmsnorm_fwd(x, w, EPS, r, want_e4m3=True)
    a = eas.rmsnorm_fwd(x, w, EPS, r, want_y=False, want_e4m3=True, want_sum=False)
    assert a[0] is None and a[3] is None and torch.equal(a[1], q) and torch.equal(a[2], scale)
    b = eas.rmsnorm_fwd(x, w, EPS, r)
    assert b[1] is None and torch.equal(b[0], y) and torch.equal(b[3], s)


@pytest.mark.parametrize("R,H", [(4, 64), (0, 64), (3, 1003), (2, 40001)])
def test_status_word_is_cleared(R, H):
    x, w, _, _ = problem(max(R, 1), H, "bf16", False, None)
    ws = torch.full((eas.rmsnorm_bwd_workspace_size(R, H),), 255, dtype=torch.uint8, device="cuda")
    eas.rmsnorm_bwd(x[:R], x[:R], w, ws=ws)
    assert eas.read_device_status(ws) == 0


def test_refusals():
    x, w, r, m = problem(4, 64, "bf16", True, "some")
    with pytest.raises(ValueError):
        eas.rmsnorm_fwd(x.t(), w)                                   # not contiguous
    with pytest.raises(ValueError):
        eas.rmsnorm_fwd(x, w[:32])
    with pytest.raises(TypeError):
        eas.rmsnorm_fwd(x, w.float())
    with pytest.raises(TypeError):
        eas.rmsnorm_fwd(x.half(), w.half())
    with pytest.raises(ValueError):
        eas.rmsnorm_fwd(x, w, residual=r[:2])
    with pytest.raises(TypeError):
        eas.rmsnorm_fwd(x, w, mask=m.bool())
    with pytest.raises(ValueError):
        eas.rmsnorm_bwd(x, r, w, mask=m[:2])
    with pytest.raises(eas.EasError, match="eps"):
        eas.rmsnorm_fwd(x, w, 0.0)
    with pytest.raises(eas.EasError, match="aligned"):
        eas.rmsnorm_fwd(torch.zeros(4 * 63 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 63), w[:63].clone())
    with pytest.raises(eas.EasError, match="workspace"):
        eas.rmsnorm_bwd(x, r, w, ws=eas.workspace(256, "cuda"))


def test_writes_stay_inside_their_buffers():
    from test_gpu_9_guard import Guarded
    for R, H, dtype in ((5, 1003, "bf16"), (33, 320, "fp32"), (3, 40001, "bf16"), (600, 64, "bf16"),
                        (2, 4096, "bf16")):
        x, w, r, m = problem(R, H, dtype, True, "some", seed=H)
        gd, dt = Guarded(x.device), DT[dtype]
        out = (gd.view((R, H), dt), gd.view((R, H), torch.uint8), gd.view((R,), torch.float32),
               gd.view((R, H), dt))
        eas.rmsnorm_fwd(x, w, EPS, r, m, want_e4m3=True, out=out)
        check_fwd(x, w, r, m, *out)
        eas.rmsnorm_bwd(x, r, w, EPS, x, m, ws=gd.bytes(eas.rmsnorm_bwd_workspace_size(R, H)),
                        dx=gd.view((R, H), dt), dweight=gd.view((H,), torch.float32))
        gd.check()


def test_autograd():
    """The wrapper's gradients, with a broadcast upstream gradient and one that
    starts off a 16-byte boundary."""
    x, w, r, m = problem(6, 100, "fp32", True, "some", seed=2)
    for t in (x, w, r):
        t.requires_grad_()
    y, s, q, scale = eas.fused_rmsnorm(x, w, r, EPS, m, want_e4m3=True)
    assert not q.requires_grad and not scale.requires_grad
    g = torch.randn(601, device="cuda")[1:].view(6, 100)
    ((y * g).sum() + s.sum()).backward()
    rdx, rdw = oracle.rmsnorm_grad(f64(g), f64(s.detach()), f64(w.detach()), EPS, np.ones((6, 100)), f64(m))
    for got, want in ((x.grad, rdx), (r.grad, rdx), (w.grad, rdw)):
        np.testing.assert_allclose(f64(got), want, rtol=1e-5, atol=1e-5)
    x2 = x.detach().clone().requires_grad_()
    y2, none, _, _ = eas.fused_rmsnorm(x2, w.detach())
    assert none is None
    y2.sum().backward()                                   # an expanded gradient
    want, _ = oracle.rmsnorm_grad(np.ones((6, 100)), f64(x2.detach()), f64(w.detach()), EPS)
    np.testing.assert_allclose(f64(x2.grad), want, rtol=1e-5, atol=1e-5)
    x3 = x.detach().clone().requires_grad_()
    _, s3, _, _ = eas.fused_rmsnorm(x3, w.detach(), r.detach())
    s3.sum().backward()                                   # only the sum is used
    assert (x3.grad == 1).all()


def test_second_derivatives_are_refused():
    x, w, _, _ = problem(3, 64, "fp32", False, None)
    x.requires_grad_()
    y, _, _, _ = eas.fused_rmsnorm(x, w)
    g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_other_stream_and_graph():
    x, w, r, m = problem(64, 1024, "bf16", True, "some", seed=8)
    want = eas.rmsnorm_fwd(x, w, EPS, r, m, want_e4m3=True)
    gx = eas.rmsnorm_bwd(x, r, w, EPS, None, m)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = eas.rmsnorm_fwd(x, w, EPS, r, m, want_e4m3=True)
    st.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = eas.rmsnorm_fwd(x, w, EPS, r, m, want_e4m3=True)
        cgx = eas.rmsnorm_bwd(x, r, w, EPS, None, m)
    for t in cap + cgx:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(cap + cgx, want + gx):
        assert torch.equal(a, b)


def test_feeds_the_e4m3_lm_head():
    """Norm with codes -> e4m3 forward -> e4m3 backward -> norm backward."""
    T, H, V = 300, 256, 500
    x, w, r, m = problem(T, H, "bf16", True, "some", seed=12)
    weight = rows((V, H), "bf16", 13, 0.2)
    t = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    y, q, scale, s = eas.rmsnorm_fwd(x, w, EPS, r, m, want_e4m3=True)
    wq, wsc = eas.quantize_rows_e4m3(weight)
    spans, ns = eas.build_active_spans(m)
    lp, ent, lse = eas.lmhead_fwd_fp8(q, scale, wq, wsc, t, m, spans, ns)
    ref, _, _ = oracle.lmhead_forward(oracle.dequantize_rows_e4m3(q.cpu().numpy(), scale.cpu().numpy()),
                                      oracle.dequantize_rows_e4m3(wq.cpu().numpy(), wsc.cpu().numpy()),
                                      t.cpu().numpy(), m.cpu().numpy())
    assert np.abs(f64(lp) - ref).max() <= 2e-3
    g = torch.ones(T, device="cuda")
    dh, _ = eas.lmhead_bwd_fp8(g, torch.zeros_like(g), y, weight, q, scale, wq, wsc, t, m, spans, ns,
                               lse, ent)
    dx, dw = eas.rmsnorm_bwd(dh, s, w, EPS, mask=m)
    assert (dx[m == 0] == 0).all() and torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_offsets_beyond_32_bits():
    """2^31 + elements: the last rows of a large call equal a small call's."""
    H, R = 8192, (1 << 18) + 3
    x = torch.full((R, H), 0.5, dtype=torch.bfloat16, device="cuda")
    tail = rows((4, H), "bf16", 1)
    x[-4:] = tail
    w = rows((H,), "bf16", 2)
    want = eas.rmsnorm_fwd(tail, w, EPS, want_e4m3=True)
    y, q, scale, _ = eas.rmsnorm_fwd(x, w, EPS, want_e4m3=True)
    assert torch.equal(y[-4:], want[0]) and torch.equal(q[-4:], want[1])
    assert torch.equal(scale[-4:], want[2])
    dx, _ = eas.rmsnorm_bwd(y, x, w, EPS)
    small, _ = eas.rmsnorm_bwd(want[0], tail, w, EPS)
    assert torch.equal(dx[-4:], small)
