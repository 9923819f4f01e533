"""The operators around the LM head where a launch gives each of its groups several
rows, tokens or chunks: sizes are taken from the machine's SM count.

Rows are independent of each other and their arithmetic does not depend on how
many a launch takes, so a large call is compared to the bit with the same rows in
small calls (which the other tests compare with 64 bits), and a sample of it with
the oracle.  Integers keep the embedding's sums exact."""
import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
from test_gpu_a_norm import DT, EPS, HALF, chain, check_fwd

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def rows(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(DT[dtype])


def masks(R, seed):
    """Single rows, and long stretches of either kind."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = torch.rand(R, device="cuda", generator=g) < 0.6
    m[R // 4:R // 3], m[R // 2:R // 2 + R // 7] = False, True
    return m.to(torch.uint8)


# ------------------------------------------------------------------- the norm

# rows within warps take several from 256 rows an SM on, rows of a CTA from 32
NARROW = [(33, 64 * 8), (128, 64 * 8), (320, 64 * 8), (333, 64 * 8), (64, 16 * 32 * 8)]
WIDE = [(1003, 64), (1088, 128), (4096, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,per_sm", NARROW + WIDE)
def test_forward_in_batches(H, per_sm, dtype):
    R, step = per_sm * sms() + 5, 4000       # 4000 rows: a batch of one, and 16-byte aligned starts
    x, r, w = rows((R, H), dtype, H), rows((R, H), dtype, H + 1, 2.0), rows((H,), dtype, H + 2)
    m = masks(R, H)
    for residual, mask, want_sum in ((True, True, True), (True, True, False), (True, False, True),
                                     (False, True, True), (False, False, True)):
        def call(a, b):
            return eas.rmsnorm_fwd(x[a:b], w, EPS, r[a:b] if residual else None, m[a:b] if mask else None,
                                   want_e4m3=True, want_sum=want_sum)
        whole = call(0, R)
        for a in range(0, R, step):
            for name, got, want in zip(("y", "codes", "scale", "s"), whole, call(a, min(a + step, R))):
                if got is not None:
                    assert torch.equal(got[a:a + step], want), (name, a, residual, mask)
        some = torch.randperm(R, generator=torch.Generator().manual_seed(1))[:97].cuda()
        y, q, scale, s = (None if t is None else t[some] for t in whole)
        check_fwd(x[some], w, r[some] if want_sum and residual else None, m[some] if mask else None,
                  *((y, q, scale, s) if want_sum or not residual else (None, None, None, None)))


# a group (a CTA, or each of its 8 warps) lists 512 rows at a time: (H, dtype, CTAs
# an SM, groups a CTA); a launch has 1024 CTAs at most
SEGMENTS = [(4096, "bf16", 2, 1), (4096, "fp32", 1, 1), (64, "bf16", 2, 8), (33, "bf16", 2, 8), (1003, "bf16", 8, 1)]


@pytest.mark.parametrize("H,dtype,per_sm,groups", SEGMENTS)
def test_backward_over_several_lists(H, dtype, per_sm, groups):
    ctas = min(per_sm * sms(), 1024)
    n_groups = ctas * groups
    R, step = 512 * n_groups + 77, 40000
    s, dy, ds, w = rows((R, H), dtype, 1, 2.0), rows((R, H), dtype, 2, 0.1), rows((R, H), dtype, 3), rows((H,), dtype, 4)
    m = masks(R, 5)
    for with_ds, mask in ((True, True), (False, True), (True, False), (False, False)):
        def call(a, b):
            return eas.rmsnorm_bwd(dy[a:b], s[a:b], w, EPS, ds[a:b] if with_ds else None, m[a:b] if mask else None)
        dx, dw = call(0, R)
        ref, absum = (torch.zeros(H, dtype=torch.float64, device="cuda") for _ in range(2))
        for a in range(0, R, step):
            assert torch.equal(dx[a:a + step], call(a, min(a + step, R))[0]), (a, with_ds, mask)
            S, D = s[a:a + step].double(), dy[a:a + step].double()
            n = S / (S.square().mean(1, keepdim=True) + EPS).sqrt()
            if mask:
                D = D * m[a:a + step, None]
            ref += (D * n).sum(0)
            absum += (D * n).abs().sum(0)
        # a group adds its rows one after the other, a CTA its groups (and the rows that a
        # warp holds abreast), a column of partial sums goes to 16 warps, and those are
        # added up; each term has rstd's error and a few roundings
        k = -(-R // n_groups) + groups + 4 + ctas / 16 + 16 + chain(H) / 2 + 8
        assert ((dw.double() - ref).abs() <= k * 2.0 ** -24 * absum).all(), (with_ds, mask)
        again = call(0, R)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


# -------------------------------------------------------------- the embedding

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,rows_abreast", [(64, 8), (1003, 1), (1088, 1), (4096, 1)])
def test_lookup_of_four_rows_a_thread(H, rows_abreast, dtype):
    """From 32 rows an SM (and as many abreast as a CTA holds) a thread takes four:
    ends that are no multiple of four, padding and a bad id inside a group."""
    from test_gpu_9_guard import Guarded
    V = 777
    table = rows((V, H), dtype, H)
    for tail in (1, 2, 3):
        T = 4 * rows_abreast * 8 * sms() + tail
        ids = np.random.default_rng(T).integers(0, V, T).astype(np.int32)
        ids[np.random.default_rng(T + 1).random(T) < 0.1] = -1
        bad = T - 6
        for at in (None, bad):
            if at is not None:
                ids[at] = V
            i = torch.from_numpy(ids).cuda()
            g = Guarded(i.device)
            ws = g.bytes(16)
            out = eas.embed_fwd(i, table, 1.75, ws=ws, out=g.view((T, H), DT[dtype]))
            assert eas.read_device_status(ws) == (0 if at is None else 1)
            real = (i >= 0) & (i < V)
            want = torch.where(real[:, None], (table[i.clamp(0, V - 1).long()].float() * 1.75), 0.0).to(DT[dtype])
            assert torch.equal(out, want)
            g.check()


def numbered(T, H, dtype):
    """A small integer for each token and column, exact in bf16."""
    t = torch.arange(T, device="cuda", dtype=torch.int64)[:, None]
    c = torch.arange(H, device="cuda", dtype=torch.int64)[None, :]
    return ((t * 2654435761 + c * 40503 >> 7) % 251 - 125).to(DT[dtype])


# chunks of 32, 64 and 128 tokens, and the sort over several launches
@pytest.mark.parametrize("T,H,V,kind,dtype", [
    (50001, 8, 152064, "padded", "bf16"), (131073, 8, 152064, "padded", "bf16"),
    (131073, 8, 900, "zipf", "bf16"), (262144 + 77, 24, 152064, "zipf", "fp32"),
    (262144 + 77, 8, 50, "uniform", "bf16"), (600000, 8, 152064, "padded", "bf16"),
    (600000, 8, 40, "uniform", "bf16"), (600000, 5, 3000, "zipf", "bf16"),
    (131073, 1003, 3000, "zipf", "bf16"), (40001, 1088, 129, "zipf", "fp32")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_every_token_finds_its_row(T, H, V, kind, dtype, accumulate):
    from test_gpu_b_embed import make_ids
    ids = torch.from_numpy(make_ids(T, V, kind, seed=5)).cuda()
    dout = numbered(T, H, dtype)
    base = (torch.arange(V * H, device="cuda").view(V, H) % 17).float()
    dw = eas.embed_bwd(ids, dout, V, 1.0, accumulate, dweight=base.clone())
    ref = torch.zeros(V, H, dtype=torch.float64, device="cuda")
    ref.index_add_(0, ids[ids >= 0].long(), dout[ids >= 0].double())
    if accumulate:
        ref += base
    assert float(ref.abs().max()) < 2 ** 24            # exact in fp32
    assert torch.equal(dw.double(), ref)
    assert torch.equal(eas.embed_bwd(ids, dout, V, 1.0, accumulate, dweight=base.clone()), dw)


def test_long_runs_of_random_values_repeat():
    """Runs of one to thousands of tokens whose sums do round: the same bits again."""
    from test_gpu_b_embed import check_bwd, make_ids
    T, H, V = 262144 + 77, 24, 3000
    ids = make_ids(T, V, "zipf", seed=2)
    i, dout = torch.from_numpy(ids).cuda(), rows((T, H), "bf16", 3)
    dw = eas.embed_bwd(i, dout, V, 1.5)
    check_bwd(ids, dout, V, 1.5, dw)
    for _ in range(3):
        assert torch.equal(eas.embed_bwd(i, dout, V, 1.5), dw)
