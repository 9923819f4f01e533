"""The global gradient norm and clipping against the oracle in 64 bits.

Tolerances.  Squares are added in fp32 over the 8 elements of a load at most
(8 roundings of 2^-24, halved by the root) and in fp64 beyond; the norm is
rounded to fp32 once and the factor is two fp32 operations, so a scaled value
is within 8 2^-24 and half a step of its type."""
import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
import oracle

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
K = 8 * 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return t.double().cpu().numpy()


def rand(n, dtype, seed, scale=1.0, off=0):
    """n values starting `off` elements past a 256-byte boundary."""
    x = torch.randn(n + off, generator=torch.Generator().manual_seed(seed)) * scale
    return x.to(DT[dtype]).cuda()[off:]


def check(grads, outs, norm, max_norm):
    rn, ro = oracle.clip_grads([f64(g) for g in grads], max_norm)
    assert abs(float(norm) - rn) <= K * rn
    for o, r in zip(outs, ro):
        assert (np.abs(f64(o) - r) <= (HALF[o.dtype] + K) * np.abs(r)).all()


LISTS = {
    "one": [(1, "fp32", 0)],
    "odd": [(1003, "bf16", 0), (7, "fp32", 0), (16384, "bf16", 0), (16385, "fp32", 0), (1, "bf16", 0)],
    "offset": [(1000, "bf16", 1), (1001, "bf16", 7), (999, "fp32", 1), (20000, "fp32", 3), (5, "bf16", 3)],
    "many": [(3 + 17 * i, "bf16" if i % 3 else "fp32", i % 5) for i in range(30)],
    "large": [(1 << 22, "fp32", 0), ((1 << 21) + 9, "bf16", 0)],
}


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0])
def test_in_place(name, max_norm):
    grads = [rand(n, d, i, 0.1, off) for i, (n, d, off) in enumerate(LISTS[name])]
    before = [g.clone() for g in grads]
    norm = eas.clip_grad_norm(grads, max_norm)
    check(before, grads, norm, max_norm)
    if max_norm == 1e9:
        assert all(torch.equal(a, b) for a, b in zip(before, grads))


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_into_other_buffers(name, max_norm):
    grads = [rand(n, d, i, 0.1, off) for i, (n, d, off) in enumerate(LISTS[name])]
    keep = [g.clone() for g in grads]
    outs = [torch.full((n + 2,), float("nan"), dtype=torch.bfloat16 if i % 2 else torch.float32,
                       device="cuda")[i % 3:i % 3 + n] for i, (n, _, _) in enumerate(LISTS[name])]
    norm = eas.clip_grad_norm(grads, max_norm, out=outs)
    check(grads, outs, norm, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(keep, grads))


def test_thousands_of_tensors():
    flat = rand(4000 * 65, "bf16", 0)
    grads = [flat[65 * i:65 * i + 65] for i in range(4000)]
    keep = flat.clone()
    norm = eas.clip_grad_norm(grads, 1.0)
    check([keep], [flat], norm, 1.0)


def test_norm_alone_and_repeats():
    grads = [rand(100003, "bf16", 1), rand(70001, "fp32", 2)]
    keep = [g.clone() for g in grads]
    a, b = eas.clip_grad_norm(grads, None), eas.clip_grad_norm(grads, None)
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(keep, grads))
    assert abs(float(a) - oracle.clip_grads([f64(g) for g in grads], 1.0)[0]) <= K * float(a)


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e17, 1e25, 1e36])
def test_squares_beyond_fp32(scale):
    grads = [rand(5000, "fp32", 1, scale), rand(3001, "bf16", 2, scale)]
    norm = eas.clip_grad_norm(grads, None)
    rn, _ = oracle.clip_grads([f64(g) for g in grads], 1.0)
    assert abs(float(norm) - rn) <= K * rn


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [0, 3, 4999])
def test_non_finite_gradients_are_left_alone(bad, at):
    for dtype in ("bf16", "fp32"):
        g = [rand(5000, dtype, 1), torch.zeros(100, device="cuda")]
        g[0][at] = bad
        keep = g[0].clone()
        norm = eas.clip_grad_norm(g, 1.0)
        assert not torch.isfinite(norm).any()
        assert torch.equal(g[0].nan_to_num(5.0), keep.nan_to_num(5.0))
        z = torch.zeros(16, device="cuda")
        z[2] = bad                                    # the only value of its load that is not zero
        assert not torch.isfinite(eas.clip_grad_norm([z], None)).any()


def test_status_word_is_cleared():
    g = rand(1000, "fp32", 0)
    ws = torch.full((eas.clip_grad_norm_workspace_size(1),), 255, dtype=torch.uint8, device="cuda")
    eas.clip_grad_norm([g], 1.0, ws=ws)
    assert eas.read_device_status(ws) == 0
    ws.fill_(255)
    eas.clip_grad_norm([g], None, ws=ws)
    assert eas.read_device_status(ws) == 0


def test_zeros_and_empty_tensors():
    z = [torch.zeros(1000, device="cuda"), torch.empty(0, device="cuda", dtype=torch.bfloat16)]
    assert float(eas.clip_grad_norm(z, 1.0)) == 0 and (z[0] == 0).all()
    assert float(eas.clip_grad_norm([z[1]], 1.0)) == 0


def test_refusals():
    g = rand(64, "fp32", 0)
    with pytest.raises(TypeError):
        eas.clip_grad_norm([g.half()], 1.0)
    with pytest.raises(ValueError):
        eas.clip_grad_norm([g[::2]], 1.0)
    with pytest.raises(ValueError):
        eas.clip_grad_norm([g], 1.0, out=[g[:32]])
    with pytest.raises(eas.EasError, match="overlaps"):
        eas.clip_grad_norm([g, g], 1.0)
    with pytest.raises(eas.EasError, match="overlaps"):
        eas.clip_grad_norm([g[:40], g[20:]], 1.0)
    with pytest.raises(eas.EasError, match="max_norm"):
        eas.clip_grad_norm([g], -1.0)
    with pytest.raises(eas.EasError, match="workspace"):
        eas.clip_grad_norm([g], 1.0, ws=eas.workspace(256, "cuda"))


def test_writes_stay_inside_their_buffers():
    from test_gpu_9_guard import Guarded
    gd = Guarded(torch.device("cuda", 0))
    grads = [gd.view((n,), DT[d]) for n, d, _ in LISTS["odd"]]
    outs = [gd.view((n,), torch.bfloat16) for n, _, _ in LISTS["odd"]]
    for i, g in enumerate(grads):
        g.copy_(rand(g.numel(), "fp32", i))
    norm = eas.clip_grad_norm(grads, 0.5, out=outs, norm=gd.view((1,), torch.float32),
                              ws=gd.bytes(eas.clip_grad_norm_workspace_size(len(grads))))
    check(grads, outs, norm, 0.5)
    eas.clip_grad_norm(grads, 0.5)
    gd.check()


def test_other_stream_and_graph():
    grads = [rand(40000, "bf16", 1), rand(3001, "fp32", 2)]
    outs, cap = [[torch.empty_like(g) for g in grads] for _ in range(2)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        norm = eas.clip_grad_norm(grads, 1.0, out=outs)
    st.synchronize()
    check(grads, outs, norm, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cnorm = eas.clip_grad_norm(grads, 1.0, out=cap)
    for c in cap:
        c.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cnorm, norm) and all(torch.equal(a, b) for a, b in zip(cap, outs))


def test_offsets_beyond_32_bits():
    n = (1 << 31) + 5
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-1], g[0] = 3.0, 4.0
    norm = eas.clip_grad_norm([g], 1.0)
    assert float(norm) == 5.0 and abs(float(g[-1]) - 0.6) < 2 ** -8 and abs(float(g[0]) - 0.8) < 2 ** -8
