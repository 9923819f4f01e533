"""The orthogonalised update against the oracle in 64 bits.

Tolerances, of the update's 2-norm.  Its rounding to bf16 is 2^-8 at worst and 2^-8 /
sqrt(3) = 2.3e-3 in the mean.  In each step four fp16 roundings of 2^-11 / sqrt(3) in
the mean (X's upper half in two products, Q, the polynomial) act on terms of |b| s^2 +
|c| s^4, together at most about twice X: sqrt(5 * 4) * 2.8e-4 * 2 = 2.5e-3 over five
steps, independent of each other.  Twice their root sum of squares, 3.4e-3, is
allowed.  A momentum in fp32 carries three roundings of its parts."""
import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
import oracle

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
FRO = 6.8e-3
ABC = eas.NEWTON_SCHULZ


def f64(t):
    return t.double().cpu().numpy()


def gradient(L, n, m, dtype, seed=0, kind="lowrank", scale=1e-3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((L, n, m), generator=g)
    if kind == "lowrank":
        r = max(1, min(16, n, m))
        s = torch.logspace(0, -1.5, r)
        x = 0.1 * x + (torch.randn((L, n, r), generator=g) * s) @ torch.randn((L, r, m), generator=g)
    return (x * scale).to(DT[dtype]).cuda()


def check(got, ref, fro=FRO):
    ref = np.asarray(ref)
    assert np.linalg.norm(f64(got) - ref) <= fro * np.linalg.norm(ref) + 1e-30


def check_all(got, grads, coeffs=(ABC,) * 5, eps=1e-7, scale=1.0, fro=FRO):
    got = got if got.dim() == 3 else got[None]
    for i in range(len(grads)):
        check(got[i], scale * oracle.orthogonalize(grads[i], coeffs, eps), fro)


# a single value, rows, columns, tiles of 128 with odd ends, both ways round
SHAPES = [(1, 1), (1, 7), (9, 1), (5, 3), (3, 5), (64, 64), (33, 200), (200, 33), (128, 128), (129, 257),
          (257, 129), (128, 1000), (700, 300), (777, 1003), (1003, 777), (100, 512), (513, 128), (128, 449),
          (384, 127)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,m", SHAPES)
def test_orthogonalize(n, m, dtype):
    for kind in ("normal", "lowrank"):
        g = gradient(1, n, m, dtype, n + m, kind)[0]
        keep = g.clone()
        out = eas.orthogonalize(g)
        assert out.dtype == torch.bfloat16 and out.shape == (n, m) and torch.equal(g, keep)
        check_all(out, f64(g)[None])


# stacks: small ones, and large enough for 256 x 256 tiles (odd ends, both ways round)
@pytest.mark.parametrize("L,n,m", [(3, 40, 70), (5, 130, 90), (12, 128, 128), (16, 520, 1100), (20, 700, 513),
                                   (40, 300, 257), (1, 3400, 3333), (2, 640, 4097),
                                   (30, 256, 512), (12, 200, 2000), (1, 1700, 1650)])
def test_stacks(L, n, m):
    g = gradient(L, n, m, "bf16", L)
    out = eas.orthogonalize(g)
    pick = range(L) if L < 10 else (0, 1, L - 1)
    for i in pick:
        check_all(out[i], f64(g[i])[None])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mom", ["bf16", "fp32"])
@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("L,n,m", [(1, 100, 60), (3, 65, 131), (2, 256, 256)])
def test_momentum(L, n, m, nesterov, mom, dtype):
    g = gradient(L, n, m, dtype, 3)
    buf = gradient(L, n, m, mom, 4, scale=3e-4)
    keep = buf.clone()
    new, u = oracle.momentum_update(f64(g), f64(buf), 0.9, nesterov)
    other = torch.full_like(buf, float("nan"))
    out = eas.muon_update(g, buf, 0.9, nesterov, new_momentum=other)
    check_all(out, u)
    assert torch.equal(buf, keep)
    half = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}[mom]
    parts = 0.9 * np.abs(f64(buf)) + 0.1 * np.abs(f64(g))
    # beta and 1 - beta round to fp32 too
    assert (np.abs(f64(other) - new) <= half * np.abs(new) + 4 * 2.0 ** -24 * parts).all()
    again = eas.muon_update(g, buf, 0.9, nesterov)          # in place
    assert torch.equal(again, out) and torch.equal(buf, other)


@pytest.mark.parametrize("shape", [(1, 129, 8000), (1, 8000, 129), (1, 200, 3001), (1, 64, 1279), (1, 64, 1280),
                                   (1, 700, 2049), (2, 300, 2500), (5, 100, 5000), (30, 128, 900), (1, 20000, 128), (1, 1, 6000), (1, 1920, 255), (1, 513, 1281)])
def test_few_long_products(shape):
    """A's tiles in parts along k: as good as in one, and the same again in the same workspace."""
    g = torch.randn(shape, generator=torch.Generator().manual_seed(5)).cuda()
    ws = eas.workspace(eas.orthogonalize_workspace_size(*shape), g.device)
    ws.fill_(0xff)
    first = eas.orthogonalize(g, ws=ws)
    check_all(first, f64(g))
    for _ in range(5):
        assert torch.equal(eas.orthogonalize(g, ws=ws), first)


def test_graphs_share_a_workspace():
    """Two captured calls over one workspace, replayed in turn: parts and counters of the one
    are nothing to the other."""
    shapes = [(1, 129, 8000), (2, 300, 2500)]
    gs = [torch.randn(s, generator=torch.Generator().manual_seed(i)).cuda() for i, s in enumerate(shapes)]
    refs = [eas.orthogonalize(g) for g in gs]
    ws = eas.workspace(max(eas.orthogonalize_workspace_size(*s) for s in shapes), "cuda:0")
    outs = [torch.empty_like(r) for r in refs]
    graphs = []
    for g, o in zip(gs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            eas.orthogonalize(g, ws=ws, out=o)
    for i in (0, 1, 1, 0, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], refs[i])


def test_steps_coefficients_scale():
    g = gradient(1, 200, 300, "fp32", 1, "normal")[0]
    for steps in (1, 2, 7):
        check_all(eas.orthogonalize(g, steps), f64(g)[None], (ABC,) * steps)
    each = [(3.0, -3.0, 1.0), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)]
    check_all(eas.orthogonalize(g, 3, each, scale=-0.2), f64(g)[None], each, scale=-0.2)
    check_all(eas.orthogonalize(g, eps=0.5), f64(g)[None], eps=0.5)


def test_orthogonal_and_ill_conditioned():
    q, _ = torch.linalg.qr(torch.randn(256, 256, generator=torch.Generator().manual_seed(0), dtype=torch.float64))
    u = eas.orthogonalize(q.float().contiguous().cuda(), 9, (1.5, -0.5, 0.0))     # 1/16 to 1 in about seven steps
    check(u, q.numpy())
    s = torch.logspace(0, -4, 256, dtype=torch.float64)
    g = (q * s) @ torch.linalg.qr(torch.randn(256, 256, dtype=torch.float64))[0]
    g = g.float().contiguous().cuda()
    check_all(eas.orthogonalize(g), f64(g)[None])


@pytest.mark.parametrize("scale", [1e-4, 1.0, 1e10, 1e17, 1e22, 1e34])
def test_magnitudes(scale):
    g = gradient(1, 90, 130, "fp32", 2, scale=scale)[0]
    check_all(eas.orthogonalize(g, eps=1e-20), f64(g)[None], eps=1e-20)
    g = g.bfloat16()
    check_all(eas.orthogonalize(g, eps=1e-20), f64(g)[None], eps=1e-20)


def test_below_eps_and_zero():
    z = torch.zeros(3, 50, 40, device="cuda")
    assert (eas.orthogonalize(z) == 0).all()
    z[1] = gradient(1, 50, 40, "fp32", 1)[0]
    out = eas.orthogonalize(z)
    assert (out[0] == 0).all() and (out[2] == 0).all()
    check_all(out[1], f64(z[1])[None])
    tiny = gradient(1, 50, 40, "fp32", 1, scale=1e-12)[0]
    ref = oracle.orthogonalize(f64(tiny), (ABC,) * 5, 1e-7)
    assert np.abs(f64(eas.orthogonalize(tiny)) - ref).max() <= 1e-2 * np.abs(ref).max()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_stays_in_its_matrix(bad):
    g = gradient(3, 140, 150, "fp32", 1)
    ref = eas.orthogonalize(g)
    g[1, 7, 9] = bad
    out = eas.orthogonalize(g)
    assert torch.isnan(out[1]).all() and torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])


@pytest.mark.parametrize("n,m", [(50, 64), (64, 50), (33, 45)])
def test_tensors_off_their_vectors(n, m):
    flat = torch.empty(2 * n * m + 8, device="cuda")
    for off in (1, 2, 3):
        g = flat.bfloat16()[off:off + n * m].view(n, m)
        g.copy_(gradient(1, n, m, "bf16", off)[0])
        buf = flat.clone()[off:off + n * m].view(n, m)
        buf.copy_(gradient(1, n, m, "fp32", 9)[0])
        out = torch.empty(n * m + 8, dtype=torch.bfloat16, device="cuda")[off:off + n * m].view(n, m)
        _, u = oracle.momentum_update(f64(g), f64(buf), 0.95, True)
        assert eas.muon_update(g, buf, out=out) is out
        check(out, oracle.orthogonalize(u, (ABC,) * 5, 1e-7))


def test_writes_stay_inside_their_buffers():
    from test_gpu_9_guard import Guarded
    for L, n, m in ((1, 777, 203), (3, 70, 130), (2, 500, 99), (16, 520, 1100), (20, 700, 513)):
        gd = Guarded(torch.device("cuda", 0))
        g, buf = gd.view((L, n, m), torch.float32), gd.view((L, n, m), torch.bfloat16)
        g.copy_(gradient(L, n, m, "fp32", 1))
        buf.copy_(gradient(L, n, m, "bf16", 2))
        ws = gd.bytes(eas.orthogonalize_workspace_size(L, n, m))
        out = gd.view((L, n, m), torch.bfloat16)
        u = oracle.momentum_update(f64(g[0]), f64(buf[0]), 0.95, True)[1]
        eas.muon_update(g, buf, ws=ws, out=out)
        assert eas.read_device_status(ws) == 0
        check_all(out[0], u[None])
        gd.check()


def test_repeats_other_stream_and_graph():
    g = gradient(4, 300, 500, "bf16", 1)
    buf = [gradient(4, 300, 500, "fp32", 2) for _ in range(3)]
    out = [None] * 3
    out[0] = eas.muon_update(g, buf[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        out[1] = eas.muon_update(g, buf[1])
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = buf[2].clone()
    with torch.cuda.graph(graph):
        out[2] = eas.muon_update(g, buf[2])
    out[2].zero_()
    buf[2].copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
    assert torch.equal(buf[0], buf[1]) and torch.equal(buf[0], buf[2])


def test_a_matrix_of_a_stack_is_as_alone():
    """The same tiles in the same order, whatever else runs beside them."""
    g = gradient(6, 150, 140, "bf16", 5)
    out = eas.orthogonalize(g)
    for i in range(6):
        assert torch.equal(out[i], eas.orthogonalize(g[i].clone()))


def test_empty_and_refusals():
    g = gradient(2, 8, 16, "fp32")
    assert eas.orthogonalize(g[:0]).shape == (0, 8, 16)
    buf = torch.zeros_like(g)
    for call, err in (
            (lambda: eas.orthogonalize(g.half()), TypeError),
            (lambda: eas.orthogonalize(g[0, 0]), ValueError),
            (lambda: eas.orthogonalize(g.mT), ValueError),
            (lambda: eas.orthogonalize(g[:, ::2]), ValueError),
            (lambda: eas.orthogonalize(g[:, :0]), eas.EasError),
            (lambda: eas.orthogonalize(g, steps=0), eas.EasError),
            (lambda: eas.orthogonalize(g, steps=33), eas.EasError),
            (lambda: eas.orthogonalize(g, coeffs=(1.0, 2.0)), (ValueError, TypeError)),
            (lambda: eas.orthogonalize(g, coeffs=[ABC] * 4), ValueError),
            (lambda: eas.orthogonalize(g, coeffs=(1.0, float("nan"), 0.0)), eas.EasError),
            (lambda: eas.orthogonalize(g, eps=0.0), eas.EasError),
            (lambda: eas.orthogonalize(g, scale=float("inf")), eas.EasError),
            (lambda: eas.orthogonalize(g, out=torch.empty_like(g)), TypeError),
            (lambda: eas.orthogonalize(g, ws=eas.workspace(256, "cuda")), eas.EasError),
            (lambda: eas.muon_update(g, None), ValueError),
            (lambda: eas.muon_update(g, buf[0]), ValueError),
            (lambda: eas.muon_update(g, buf, beta=1.5), eas.EasError),
            (lambda: eas.muon_update(g, g), eas.EasError),
            (lambda: eas.muon_update(g, buf, new_momentum=g), eas.EasError),
            (lambda: eas.muon_update(g, buf, new_momentum=buf.bfloat16()), TypeError)):
        with pytest.raises(err):
            call()


def test_more_elements_than_32_bits_count():
    n, m = 32770, 33000
    g = torch.empty((2, n, m), dtype=torch.bfloat16, device="cuda")
    g[0].normal_(generator=torch.Generator("cuda").manual_seed(0))
    g[1] = g[0]
    g[1, -1, -1] = 0                          # one value differs
    out = eas.orthogonalize(g, steps=1, coeffs=(2.0, 0.0, 0.0))
    for i in range(2):
        ref = 2 * g[i].float() / g[i].float().norm()
        assert float((out[i].float() - ref).norm() / ref.norm()) < FRO
        del ref
    assert float(out[1, -1, -1]) == 0 and float(out[0, -1, -1]) != 0
