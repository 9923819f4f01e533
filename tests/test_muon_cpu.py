"""Refusals of the orthogonalised update that the host sees (CPU only; no pointer here
is ever read)."""
import ctypes
import itertools
import math

import pytest
import torch

import entropy_active_span_gb300 as eas
from entropy_active_span_gb300 import _lib

BF, FP = _lib.EAS_BF16, _lib.EAS_FP32
INVALID, WORKSPACE = _lib.EAS_ERR_INVALID_ARG, _lib.EAS_ERR_WORKSPACE
L, R, C, STEPS = 2, 24, 40, 2
SIZES = {"grad": 2 * L * R * C, "mom": 4 * L * R * C, "new": 4 * L * R * C, "out": 2 * L * R * C, "ws": 0}
P = {n: (i + 1) << 24 for i, n in enumerate(SIZES)}


def call(lib, L=L, R=R, C=C, gd=BF, md=FP, beta=0.9, nesterov=1, coeffs=(3.0, -4.0, 2.0) * STEPS, steps=STEPS,
         eps=1e-7, scale=1.0, ws_bytes=1 << 40, **p):
    p = {**P, **p}
    arr = (ctypes.c_float * len(coeffs))(*coeffs) if coeffs else None
    return lib.eas_orthogonalize(p["grad"], gd, p["mom"], p["new"], md, L, R, C, beta, nesterov, arr, steps, eps,
                                 scale, p["out"], p["ws"], ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(L=-1), dict(L=65536), dict(R=0), dict(C=0), dict(R=65537), dict(C=65537), dict(L=65535, R=65536, C=65536),
    dict(gd=_lib.EAS_E4M3), dict(md=_lib.EAS_E4M3), dict(beta=-0.1), dict(beta=1.1), dict(beta=math.nan),
    dict(nesterov=2), dict(coeffs=None), dict(coeffs=(1.0, math.nan, 0.0) * STEPS),
    dict(coeffs=(1.0, 0.0, math.inf) * STEPS), dict(steps=0), dict(steps=33, coeffs=(1.0,) * 99), dict(eps=0.0),
    dict(eps=-1.0), dict(eps=math.inf), dict(scale=math.nan), dict(grad=None), dict(out=None), dict(ws=None),
    dict(mom=None), dict(new=None), dict(grad=P["grad"] + 1), dict(mom=P["mom"] + 2), dict(new=P["new"] + 2),
    dict(out=P["out"] + 1), dict(ws=P["ws"] + 64), dict(new=P["mom"] + 4), dict(gd=FP, grad=P["mom"], new=P["mom"])])
def test_refuses(libeas, bad):
    assert call(libeas, **bad) == INVALID


@pytest.mark.parametrize("eps", [1e-38, 9e-31])
def test_refuses_an_eps_whose_factor_leaves_fp32(libeas, eps):
    assert call(libeas, eps=eps) == INVALID
    assert b"eps" in libeas.eas_last_error()


def test_workspace(libeas):
    size = libeas.eas_orthogonalize_workspace_size
    assert call(libeas, ws_bytes=size(L, R, C) - 1) == WORKSPACE
    assert size(-1, 4, 4) == size(1, 0, 4) == size(1, 4, 65537) == 0
    assert size(1, 4096, 4096) >= (6 + 4) * 4096 * 4096
    assert size(0, 4, 4) > 0 and size(2, 100, 300) == size(2, 300, 100)


def test_no_output_shares_a_byte(libeas):
    sizes = {**SIZES, "ws": libeas.eas_orthogonalize_workspace_size(L, R, C)}
    for a, b in itertools.permutations(sizes, 2):
        if a not in ("new", "out", "ws"):
            continue
        for at in (P[b] + sizes[b] - 1 - (sizes[b] - 1) % 256, P[b] - (sizes[a] - 1) // 256 * 256):
            assert call(libeas, **{a: at}) == INVALID, (a, b)
            assert b"overlaps" in libeas.eas_last_error(), (a, b)


def test_binding_refuses():
    g = torch.zeros(4, 4)
    for f in (lambda: eas.orthogonalize(g), lambda: eas.muon_update(g, g)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    with pytest.raises(TypeError):
        eas.orthogonalize([1.0])
