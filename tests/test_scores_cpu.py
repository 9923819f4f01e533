"""Refusals of the scores of logits that the host sees (CPU only; no pointer here is
ever read)."""
import itertools
import math

import pytest
import torch

import entropy_active_span_gb300 as eas
from entropy_active_span_gb300 import _lib

BF, FP = _lib.EAS_BF16, _lib.EAS_FP32
INVALID, WORKSPACE = _lib.EAS_ERR_INVALID_ARG, _lib.EAS_ERR_WORKSPACE
N, V, M, K, LD = 6, 50, 3, 4, 56

SIZES = {"x": 2 * ((N - 1) * LD + V), "tok": 4 * N * M, "mask": N, "lp": 4 * N * M, "ent": 4 * N,
         "lse": 4 * N, "top": 4 * N * K, "ids": 4 * N * K, "ws": 16, "glp": 4 * N * M, "gent": 4 * N,
         "dx": 2 * ((N - 1) * LD + V)}
P = {n: (i + 1) << 20 for i, n in enumerate(SIZES)}


def fwd(lib, ld=LD, N=N, V=V, M=M, k=K, dtype=BF, scale=1.0, ws_bytes=16, **p):
    p = {**P, **p}
    return lib.eas_token_logprobs_fwd(p["x"], ld, p["tok"], p["mask"], N, V, M, k, dtype, scale, p["lp"],
                                      p["ent"], p["lse"], p["top"], p["ids"], p["ws"], ws_bytes, None)


def bwd(lib, ld=LD, ldd=LD, N=N, V=V, M=M, dtype=BF, scale=1.0, ws_bytes=16, **p):
    p = {**P, **p}
    return lib.eas_token_logprobs_bwd(p["glp"], p["gent"], p["x"], ld, p["tok"], p["mask"], p["lse"],
                                      p["ent"], N, V, M, dtype, scale, p["dx"], ldd, p["ws"], ws_bytes, None)


BAD = [dict(N=-1), dict(N=(1 << 28) + 1), dict(V=0), dict(V=1 << 31, ld=1 << 31), dict(M=-1), dict(M=129),
       dict(ld=V - 1), dict(dtype=_lib.EAS_E4M3), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
       dict(scale=math.inf), dict(x=None), dict(tok=None), dict(lse=None), dict(ent=None),
       dict(x=P["x"] + 1), dict(tok=P["tok"] + 2), dict(lse=P["lse"] + 2), dict(ent=P["ent"] + 1),
       dict(ws=P["ws"] + 8)]


@pytest.mark.parametrize("bad", BAD + [
    dict(k=-1), dict(k=65), dict(k=V + 1), dict(lp=None), dict(top=None), dict(ids=None),
    dict(lp=P["lp"] + 1), dict(top=P["top"] + 2), dict(ids=P["ids"] + 3)])
def test_forward_refuses(libeas, bad):
    assert fwd(libeas, **bad) == INVALID


@pytest.mark.parametrize("bad", BAD + [
    dict(ldd=V - 1), dict(glp=None), dict(dx=None), dict(glp=P["glp"] + 2), dict(gent=P["gent"] + 2),
    dict(dx=P["dx"] + 1), dict(dx=P["x"], ldd=LD + 1), dict(dx=P["x"] + 2 * V)])
def test_backward_refuses(libeas, bad):
    assert bwd(libeas, **bad) == INVALID


def test_workspace_too_small(libeas):
    assert fwd(libeas, ws_bytes=15) == WORKSPACE and bwd(libeas, ws_bytes=8) == WORKSPACE


@pytest.mark.parametrize("call,bufs,written", [
    (fwd, ("x", "tok", "mask", "lp", "ent", "lse", "top", "ids", "ws"), ("lp", "ent", "lse", "top", "ids", "ws")),
    (bwd, ("glp", "gent", "x", "tok", "mask", "lse", "ent", "dx", "ws"), ("dx", "ws"))])
def test_no_output_shares_a_byte(libeas, call, bufs, written):
    for a, b in itertools.permutations(bufs, 2):
        if a not in written:
            continue
        for at in (P[b] + SIZES[b] - 16 + (SIZES[b] % 16 and 16 - SIZES[b] % 16), P[b] - SIZES[a] + 16 - SIZES[a] % 16):
            at -= at % 16
            if at >= P[b] + SIZES[b] or at + SIZES[a] <= P[b]:
                continue
            assert call(libeas, **{a: at}) == INVALID, (a, b)
            assert b"overlaps" in libeas.eas_last_error(), (a, b)


def test_binding_refuses():
    x = torch.zeros(2, 8)
    ids = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: eas.token_logprobs_fwd(x, ids),
                 lambda: eas.token_logprobs_bwd(x[:, 0], None, x, ids, x[:, 0], x[:, 0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        eas.token_logprobs_fwd([1.0])
