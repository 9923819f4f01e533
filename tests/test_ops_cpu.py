"""Refusals of the operators around the LM head that the host sees: bad
arguments of the C entry points and of the binding (CPU only; no pointer here
is ever read)."""
import ctypes

import pytest
import torch

import entropy_active_span_gb300 as eas
from entropy_active_span_gb300 import _lib

P = 256          # a fake, aligned address, and others far from it
A, B, C, D, E, F = (P + (i << 20) for i in range(1, 7))
BIG = 1 << 40
INVALID, WORKSPACE = _lib.EAS_ERR_INVALID_ARG, _lib.EAS_ERR_WORKSPACE


def norm_fwd(lib, x=A, r=B, w=P, mask=P, R=4, H=64, dtype=_lib.EAS_BF16, eps=1e-6, s=C, y=D,
             q=E, scale=F):
    return lib.eas_rmsnorm_fwd(x, r, w, mask, R, H, dtype, eps, s, y, q, scale, None)


@pytest.mark.parametrize("bad", [
    dict(R=-1), dict(H=0), dict(H=(1 << 20) + 1), dict(dtype=_lib.EAS_E4M3), dict(eps=0.0),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(w=None),
    dict(q=None), dict(scale=None), dict(r=None), dict(x=A + 8), dict(r=B + 2), dict(w=P + 4),
    dict(y=D + 8), dict(q=E + 1), dict(s=C + 8), dict(s=None, y=None, q=None, scale=None),
    dict(y=A), dict(y=B + 16), dict(y=C), dict(q=A + 496), dict(q=C), dict(q=D + 16),
    dict(s=A + 64), dict(s=B - 64),
])
def test_rmsnorm_fwd_refuses(libeas, bad):
    assert norm_fwd(libeas, **bad) == INVALID


def norm_bwd(lib, dy=A, s=B, w=P, ds=C, mask=P, R=4, H=64, dtype=_lib.EAS_BF16, eps=1e-6,
             dx=D, dw=E, ws=F, ws_bytes=BIG):
    return lib.eas_rmsnorm_bwd(dy, s, w, ds, mask, R, H, dtype, eps, dx, dw, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(R=-1), dict(H=0), dict(dtype=7), dict(eps=0.0), dict(dy=None), dict(s=None), dict(w=None),
    dict(dx=None), dict(dw=None), dict(ws=None), dict(dy=A + 8), dict(s=B + 4), dict(ds=C + 8),
    dict(dx=D + 8), dict(dw=E + 4), dict(ws=F + 16), dict(dx=A), dict(dx=B + 64), dict(dx=C + 64),
])
def test_rmsnorm_bwd_refuses(libeas, bad):
    assert norm_bwd(libeas, **bad) == INVALID
    need = libeas.eas_rmsnorm_bwd_workspace_size(4, 64)
    assert norm_bwd(libeas, ws_bytes=need - 1) == WORKSPACE


def embed_fwd(lib, ids=P, table=A, T=4, H=64, V=10, dtype=_lib.EAS_BF16, scale=1.0, out=B,
              ws=C, ws_bytes=64):
    return lib.eas_embed_fwd(ids, table, T, H, V, dtype, scale, out, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(V=0), dict(V=1 << 31), dict(dtype=_lib.EAS_E4M3),
    dict(scale=float("nan")), dict(ids=None), dict(table=None), dict(out=None), dict(ids=P + 2),
    dict(table=A + 8), dict(out=B + 8), dict(ws=C + 8), dict(out=A), dict(out=A + 1264),
])
def test_embed_fwd_refuses(libeas, bad):
    assert embed_fwd(libeas, **bad) == INVALID
    assert embed_fwd(libeas, ws_bytes=8) == WORKSPACE


def embed_bwd(lib, ids=P, dout=A, T=4, H=64, V=10, dtype=_lib.EAS_BF16, scale=1.0, accumulate=0,
              dw=B, ws=C, ws_bytes=BIG):
    return lib.eas_embed_bwd(ids, dout, T, H, V, dtype, scale, accumulate, dw, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(V=0), dict(dtype=_lib.EAS_E4M3), dict(scale=float("inf")),
    dict(accumulate=2), dict(ids=None), dict(dout=None), dict(dw=None), dict(ws=None),
    dict(ids=P + 1), dict(dout=A + 8), dict(dw=B + 8), dict(ws=C + 16), dict(dw=A + 496),
])
def test_embed_bwd_refuses(libeas, bad):
    assert embed_bwd(libeas, **bad) == INVALID
    need = libeas.eas_embed_bwd_workspace_size(4, 64, 10)
    assert embed_bwd(libeas, ws_bytes=need - 1) == WORKSPACE


def clip(lib, ins, outs, numels, dts, odts, max_norm=1.0, norm=P, ws=P, ws_bytes=BIG):
    n = len(numels)
    pv, i64, i32 = ctypes.c_void_p * n, ctypes.c_int64 * n, ctypes.c_int32 * n
    return lib.eas_clip_grad_norm(pv(*ins), pv(*outs) if outs else None, i64(*numels), i32(*dts),
                                  i32(*odts), n, max_norm, norm, ws, ws_bytes, None)


BF, FP = _lib.EAS_BF16, _lib.EAS_FP32


@pytest.mark.parametrize("ins,outs,numels,dts,odts", [
    ([P], [P], [-1], [FP], [FP]),                      # a negative length
    ([P], [P], [1 << 41], [FP], [FP]),                 # beyond the chunk index
    ([P], [P], [8], [2], [FP]),                        # an unknown dtype
    ([P], [P], [8], [FP], [9]),
    ([0], [P], [8], [FP], [FP]),                       # null
    ([P], [0], [8], [FP], [FP]),
    ([P + 2], [P + 2], [8], [FP], [FP]),               # not aligned to the element
    ([P], [4 * P + 1], [8], [FP], [BF]),
    ([P], [P], [8], [FP], [BF]),                       # in place, but narrower
    ([P, P], [P, P], [8, 8], [FP, FP], [FP, FP]),      # the same tensor twice, in place
    ([P, P + 16], [P, P + 16], [8, 8], [FP, FP], [FP, FP]),      # overlapping in place
    ([P, 4 * P], [8 * P, 8 * P + 28], [8, 8], [FP, FP], [FP, FP]),   # overlapping outputs
    ([P, 4 * P], [4 * P, 8 * P], [8, 8], [FP, FP], [FP, FP]),    # an output on another's input
    ([P], [P + 16], [8], [FP], [FP]),                  # an output partly on its own input
])
def test_clip_refuses(libeas, ins, outs, numels, dts, odts):
    assert clip(libeas, ins, outs, numels, dts, odts) == INVALID


def test_clip_refuses_scalars(libeas):
    one = ([P], [P], [8], [FP], [FP])
    assert clip(libeas, *one, max_norm=-1.0) == INVALID
    assert clip(libeas, *one, max_norm=float("nan")) == INVALID
    assert clip(libeas, *one, norm=None) == INVALID
    assert clip(libeas, *one, ws=None) == INVALID
    assert clip(libeas, *one, ws=P + 8) == INVALID
    assert clip(libeas, *one, ws_bytes=64) == WORKSPACE
    assert libeas.eas_clip_grad_norm(None, None, None, None, None, -1, 1.0, P, P, BIG, None) == INVALID


def test_workspace_sizes(libeas):
    assert libeas.eas_rmsnorm_bwd_workspace_size(-1, 64) == 0
    assert libeas.eas_embed_bwd_workspace_size(4, 0, 10) == 0
    assert libeas.eas_clip_grad_norm_workspace_size(-1) == 0
    assert libeas.eas_rmsnorm_bwd_workspace_size(0, 64) > 0
    assert libeas.eas_embed_bwd_workspace_size(0, 64, 10) > 0
    assert libeas.eas_embed_bwd_workspace_size(1 << 17, 7168, 129280) > 4 * 4 * (1 << 17)
    assert libeas.eas_clip_grad_norm_workspace_size(5000) > libeas.eas_clip_grad_norm_workspace_size(1)


def test_binding_refuses_host_tensors_and_types():
    x, w = torch.zeros(2, 8), torch.ones(8)
    ids = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: eas.rmsnorm_fwd(x, w), lambda: eas.rmsnorm_bwd(x, x, w),
                 lambda: eas.embed_fwd(ids, x), lambda: eas.embed_bwd(ids, x, 4),
                 lambda: eas.clip_grad_norm([x], 1.0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        eas.rmsnorm_fwd([1.0], w)
    with pytest.raises(ValueError, match="no gradients"):
        eas.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError, match="one tensor for each"):
        eas.clip_grad_norm([x], 1.0, out=[])
