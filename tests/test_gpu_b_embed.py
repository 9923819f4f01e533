"""The embedding lookup and its gradient against the oracle in 64 bits.

Tolerances.  A looked-up value is one fp32 product and one rounding to the
type.  A gradient row of n tokens is a sum of n terms in fp32 and one product:
(n + 1) 2^-24 of the sum of the absolute terms."""
import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
import oracle

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return t.double().cpu().numpy()


def rows(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(DT[dtype]).cuda()


def make_ids(T, V, kind, seed=0):
    rng = np.random.default_rng(seed + T)
    if kind == "zipf":
        ids = np.minimum(rng.zipf(1.3, T) - 1, V - 1)
    elif kind == "one":
        ids = np.full(T, V - 1)
    else:
        ids = rng.integers(0, V, T)
    ids = ids.astype(np.int32)
    if kind in ("zipf", "padded"):
        ids[rng.random(T) < 0.2] = -1
    if kind == "padding":
        ids[:] = -1
    return ids


def check_bwd(ids, dout, V, scale, dw, base=None):
    d = f64(dout)
    sc = float(np.float32(scale))
    ref = oracle.embed_grad(ids, d, V, sc)
    absum = oracle.embed_grad(ids, np.abs(d), V, abs(sc))
    real = ids[(ids >= 0) & (ids < V)]
    n = np.bincount(real, minlength=V)[:, None]
    tol = (n + 1) * 2.0 ** -24 * absum
    if base is not None:
        ref = ref + f64(base)
        tol = tol + 2.0 ** -24 * np.abs(ref) * (n > 0)
    assert (np.abs(f64(dw) - ref) <= tol * (1 + 1e-6)).all()


SHAPES = [(1, 64, 1), (1, 1003, 10), (5, 7, 3), (16, 4096, 1500), (300, 320, 600), (512, 1003, 77), (513, 136, 77), (2049, 256, 511),
          (2048, 64, 512), (4100, 1088, 513), (9000, 136, 270000)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H,V", SHAPES)
def test_lookup(T, H, V, dtype):
    V = min(V, 5000)
    table = rows((V, H), dtype, V)
    for kind, scale in (("uniform", 1.0), ("padded", H ** 0.5)):
        ids = make_ids(T, V, kind)
        ws = eas.workspace(16, "cuda")
        out = eas.embed_fwd(torch.from_numpy(ids).cuda(), table, scale, ws=ws)
        assert eas.read_device_status(ws) == 0
        ref = oracle.embed(ids, f64(table), float(np.float32(scale)))
        assert (np.abs(f64(out) - ref) <= (HALF[table.dtype] + 2.0 ** -24) * np.abs(ref)).all()
        if scale == 1.0:
            assert torch.equal(out, table[torch.from_numpy(ids).cuda().long()])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H,V", SHAPES)
def test_gradient(T, H, V, dtype):
    dout = rows((T, H), dtype, T)
    for kind in ("uniform", "zipf", "one", "padding"):
        ids = make_ids(T, V, kind)
        i = torch.from_numpy(ids).cuda()
        dw = eas.embed_bwd(i, dout, V, 1.5, dweight=torch.full((V, H), float("nan"), device="cuda"))
        check_bwd(ids, dout, V, 1.5, dw)
        assert torch.equal(dw, eas.embed_bwd(i, dout, V, 1.5))         # repeats to the bit


@pytest.mark.parametrize("T,H,V,kind", [(700, 320, 50, "zipf"), (700, 1003, 900, "uniform"),
                                        (5000, 64, 7, "zipf"), (300, 64, 20, "padding")])
def test_accumulate(T, H, V, kind):
    dout, base = rows((T, H), "bf16", 1), rows((V, H), "fp32", 2)
    ids = make_ids(T, V, kind)
    dw = eas.embed_bwd(torch.from_numpy(ids).cuda(), dout, V, 2.0, accumulate=True, dweight=base.clone())
    check_bwd(ids, dout, V, 2.0, dw, base)
    untouched = np.setdiff1d(np.arange(V), ids)
    assert torch.equal(dw[untouched], base[untouched])


def test_a_run_across_many_chunks():
    """One id of 20000 tokens between others: pieces from several workers."""
    T, H, V = 30001, 72, 12
    ids = np.sort(np.random.default_rng(0).integers(0, V, T)).astype(np.int32)
    ids[5000:25000] = 6
    np.random.default_rng(1).shuffle(ids)
    dout = rows((T, H), "fp32", 5)
    dw = eas.embed_bwd(torch.from_numpy(ids).cuda(), dout, V)
    check_bwd(ids, dout, V, 1.0, dw)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("V", [40, 400])
def test_runs_around_chunk_boundaries(V, accumulate):
    """Runs that start, end and lie across the workers' chunks (16 tokens at this
    size, and powers of two above it) at every offset; small integers, so exact."""
    rng = np.random.default_rng(V)
    lens = rng.choice([1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 64, 80], V)
    lens[0], lens[1] = 16, 16
    ids = np.repeat(np.arange(V), lens).astype(np.int32)
    assert len(ids) > 600
    order = rng.permutation(len(ids))
    for these in (ids, ids[order], np.concatenate([ids, np.full(100, -1, np.int32)])):
        T, H = len(these), 72
        dout = torch.from_numpy(rng.integers(-4, 5, (T, H)).astype(np.float32)).bfloat16().cuda()
        base = torch.zeros(V, H, device="cuda")
        dw = eas.embed_bwd(torch.from_numpy(these).cuda(), dout, V, 1.0, accumulate, dweight=base)
        assert np.array_equal(f64(dw), oracle.embed_grad(these, f64(dout), V, 1.0))


@pytest.mark.parametrize("T", [8192, 8193, 20000, 50001, 131072, 131073, 262144 + 77, 600000])
def test_large_sorts(T):
    """The sort in one launch at each of its sizes, and beyond them over several:
    integers, so exact."""
    V, H = 152064, 8
    ids = make_ids(T, V, "padded", seed=3)
    dout = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    dw = eas.embed_bwd(torch.from_numpy(ids).cuda(), dout, V)
    count = np.bincount(ids[ids >= 0], minlength=V)
    assert np.array_equal(f64(dw), np.repeat(count[:, None], H, 1).astype(float))


def test_padding_and_bad_ids():
    V, H = 9, 64
    table = rows((V, H), "fp32", 0)
    ids = np.array([0, -1, 8, 9, 3, -2, 2 ** 31 - 1, -(2 ** 31)], np.int32)
    i, ws = torch.from_numpy(ids).cuda(), eas.workspace(64, "cuda")
    out = eas.embed_fwd(i, table, ws=ws)
    assert eas.read_device_status(ws) == 1                     # EAS_ERR_INVALID_ARG
    assert (out[[1, 3, 5, 6, 7]] == 0).all() and torch.equal(out[[0, 2, 4]], table[[0, 8, 3]])
    dout = torch.full((8, H), float("nan"), device="cuda")
    dout[[0, 2, 4]] = 1.0
    ws = eas.workspace(eas.embed_bwd_workspace_size(8, H, V), "cuda")
    dw = eas.embed_bwd(i, dout, V, ws=ws)
    assert eas.read_device_status(ws) == 1
    want = torch.zeros(V, H, device="cuda")
    want[[0, 8, 3]] = 1.0
    assert torch.equal(dw, want)                               # nothing of the bad rows is read
    ok = torch.from_numpy(np.array([0, -1, 8], np.int32)).cuda()
    eas.embed_fwd(ok, table, ws=ws)
    assert eas.read_device_status(ws) == 0                     # the next call clears the status
    eas.embed_bwd(ok, dout[:3].contiguous(), V, ws=ws)
    assert eas.read_device_status(ws) == 0


def test_no_tokens():
    ids = torch.zeros(0, dtype=torch.int32, device="cuda")
    table = rows((5, 64), "bf16", 0)
    ws = torch.full((64,), 255, dtype=torch.uint8, device="cuda")
    assert eas.embed_fwd(ids, table, ws=ws).shape == (0, 64)
    assert eas.read_device_status(ws) == 0
    dw = eas.embed_bwd(ids, table[:0], 5)
    assert (dw == 0).all()
    keep = torch.ones(5, 64, device="cuda")
    eas.embed_bwd(ids, table[:0], 5, accumulate=True, dweight=keep)
    assert (keep == 1).all()


def test_nan_and_infinity_stay_in_their_rows():
    ids = torch.tensor([0, 1, 2, 1], dtype=torch.int32, device="cuda")
    dout = torch.ones(4, 64, device="cuda")
    dout[1], dout[2] = float("nan"), float("inf")
    dw = eas.embed_bwd(ids, dout, 4)
    assert (dw[0] == 1).all() and torch.isnan(dw[1]).all() and torch.isinf(dw[2]).all() and (dw[3] == 0).all()


def test_refusals():
    table = rows((9, 64), "bf16", 0)
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        eas.embed_fwd(ids.long(), table)
    with pytest.raises(TypeError):
        eas.embed_fwd(ids, table.half())
    with pytest.raises(ValueError):
        eas.embed_fwd(ids, table.t())
    with pytest.raises(ValueError):
        eas.embed_fwd(ids[::2], table)
    with pytest.raises(ValueError):
        eas.embed_bwd(ids, table, 9)                           # 3 ids, 9 rows
    with pytest.raises(ValueError):
        eas.embed_bwd(ids, table[:3], 9, accumulate=True)      # nothing to add to
    with pytest.raises(ValueError):
        eas.embed_bwd(ids, table[:3], 9, dweight=torch.zeros(8, 64, device="cuda"))
    with pytest.raises(eas.EasError, match="scale"):
        eas.embed_fwd(ids, table, float("nan"))
    with pytest.raises(eas.EasError, match="workspace"):
        eas.embed_bwd(ids, table[:3], 9, ws=eas.workspace(256, "cuda"))


def test_writes_stay_inside_their_buffers():
    from test_gpu_9_guard import Guarded
    for T, H, V, dtype, kind in ((700, 1003, 90, "bf16", "zipf"), (5000, 320, 77, "fp32", "zipf"),
                                 (3, 64, 5, "bf16", "uniform"), (2500, 64, 1000, "bf16", "one")):
        ids = make_ids(T, V, kind)
        i = torch.from_numpy(ids).cuda()
        g = Guarded(i.device)
        eas.embed_fwd(i, rows((V, H), dtype, 1), ws=g.bytes(16), out=g.view((T, H), DT[dtype]))
        dw = g.view((V, H), torch.float32)
        dout = rows((T, H), dtype, 2)
        eas.embed_bwd(i, dout, V, ws=g.bytes(eas.embed_bwd_workspace_size(T, H, V)), dweight=dw)
        check_bwd(ids, dout, V, 1.0, dw)
        g.check()


def test_autograd():
    T, H, V = 50, 100, 30
    table = rows((V, H), "fp32", 0).requires_grad_()
    ids = make_ids(T, V, "padded")
    out = eas.fused_embedding(torch.from_numpy(ids).cuda(), table, 3.0)
    g = torch.randn(T * H + 1, device="cuda")[1:].view(T, H)
    (out * g).sum().backward()
    check_bwd(ids, g, V, 3.0, table.grad)
    table.grad = None
    eas.fused_embedding(torch.from_numpy(ids).cuda(), table).sum().backward()   # an expanded gradient
    check_bwd(ids, torch.ones(T, H), V, 1.0, table.grad)


def test_other_stream_and_graph():
    T, H, V = 3000, 256, 400
    i = torch.from_numpy(make_ids(T, V, "zipf")).cuda()
    dout, table = rows((T, H), "bf16", 0), rows((V, H), "bf16", 1)
    want, emb = eas.embed_bwd(i, dout, V), eas.embed_fwd(i, table)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = eas.embed_bwd(i, dout, V)
    st.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap, cemb = eas.embed_bwd(i, dout, V), eas.embed_fwd(i, table)
    cap.zero_()
    cemb.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap, want) and torch.equal(cemb, emb)


def test_offsets_beyond_32_bits():
    """Tables and gradients of more than 2^31 elements."""
    V, H = (1 << 18) + 5, 8192
    table = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    table[-1], table[0] = 2.0, 1.0
    ids = torch.tensor([V - 1, 0, V - 1], dtype=torch.int32, device="cuda")
    out = eas.embed_fwd(ids, table)
    assert (out[0] == 2).all() and (out[1] == 1).all() and (out[2] == 2).all()
    del table
    dw = eas.embed_bwd(ids, out, V)
    assert (dw[-1] == 4).all() and (dw[0] == 1).all() and (dw[1:-1] == 0).all()
