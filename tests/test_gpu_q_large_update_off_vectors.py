"""The larger update's kernels on a gradient, a momentum and an output that start off their
16 bytes at sizes whose rows would fit vectors.  Tolerance: what the update allows itself."""
import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
import oracle
from test_gpu_k_muon import ABC, check, f64, gradient

pytestmark = pytest.mark.gpu


def off_by(x, at):
    """A copy of x that starts `at` elements behind a 16-byte boundary."""
    flat = torch.full((x.numel() + 16,), 7.0, dtype=x.dtype, device=x.device)
    v = flat[at:at + x.numel()].view(x.shape)
    v.copy_(x)
    return flat, v


# half tiles both ways round, whole tiles, pairs
@pytest.mark.parametrize("L,n,m", [(1, 256, 512), (1, 512, 256), (30, 256, 512), (16, 520, 1104)])
@pytest.mark.parametrize("mom", [torch.bfloat16, torch.float32])
def test_off_their_vectors(L, n, m, mom):
    g, buf = gradient(L, n, m, "bf16", 1), gradient(L, n, m, "fp32", 2).to(mom)
    ref_buf = buf.clone()
    ref = eas.muon_update(g, ref_buf)
    for which in ("grad", "momentum", "new", "out", "all"):
        fg, vg = off_by(g, 1 if which in ("grad", "all") else 0)
        fb, vb = off_by(buf, 1 if which in ("momentum", "all") else 0)
        fn, vn = off_by(torch.zeros_like(buf), 3 if which in ("new", "all") else 0)
        fo, vo = off_by(torch.zeros_like(ref), 1 if which in ("out", "all") else 0)
        assert eas.muon_update(vg, vb, new_momentum=vn, out=vo) is vo
        # X is the same to the bit where the norm's sums have the same order: those of grad
        # and momentum go by their vectors
        if which in ("new", "out"):
            assert torch.equal(vo, ref)
        assert torch.equal(vn, ref_buf) and torch.equal(vb, buf)
        _, u = oracle.momentum_update(f64(vg[0]), f64(vb[0]), 0.95, True)
        check(vo[0], oracle.orthogonalize(u, (ABC,) * 5, 1e-7))
        for flat, v in ((fn, vn), (fo, vo)):
            at = v.storage_offset()
            assert (flat[:at] == 7).all() and (flat[at + v.numel():] == 7).all()
        assert np.isfinite(f64(vo[-1])).all()
