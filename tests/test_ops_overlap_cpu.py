"""Outputs and workspaces of the operators around the LM head that share a byte
with another buffer of the call are refused (CPU only; no pointer here is ever
read).  Every pair of buffers of every call is tried, with the second one ending
on, and starting on, a byte of the first."""
import ctypes
import itertools

import pytest

from entropy_active_span_gb300 import _lib

BF, FP = _lib.EAS_BF16, _lib.EAS_FP32
BIG = 1 << 40
R, H, V = 6, 64, 10


def fwd(lib, p):
    return lib.eas_rmsnorm_fwd(p["x"], p["r"], p["w"], p["mask"], R, H, BF, 1e-6, p["s"], p["y"],
                               p["q"], p["scale"], None)


def bwd(lib, p):
    return lib.eas_rmsnorm_bwd(p["dy"], p["s"], p["w"], p["ds"], p["mask"], R, H, BF, 1e-6, p["dx"],
                               p["dw"], p["ws"], BIG, None)


def look(lib, p):
    return lib.eas_embed_fwd(p["ids"], p["table"], R, H, V, BF, 1.0, p["out"], p["ws"], 64, None)


def grad(lib, p):
    return lib.eas_embed_bwd(p["ids"], p["dout"], R, H, V, BF, 1.0, 1, p["dw"], p["ws"], BIG, None)


def clip(lib, p, outs=True):
    pv, i64, i32 = ctypes.c_void_p * 2, ctypes.c_int64 * 2, ctypes.c_int32 * 2
    return lib.eas_clip_grad_norm(pv(p["a"], p["b"]), pv(p["oa"], p["ob"]) if outs else None,
                                  i64(R * H, 7), i32(BF, FP), i32(FP, BF), 2, 1.0, p["norm"], p["ws"],
                                  BIG, None)


def norm_alone(lib, p):
    return clip(lib, p, outs=False)


ROWS, ROW, CODES = 2 * R * H, 2 * H, R * H
# call: (its buffers and their bytes; 0: the workspace), those that are written
CALLS = {
    fwd: (dict(x=ROWS, r=ROWS, w=ROW, mask=R, s=ROWS, y=ROWS, q=CODES, scale=4 * R), "s y q scale"),
    bwd: (dict(dy=ROWS, s=ROWS, w=ROW, ds=ROWS, mask=R, dx=ROWS, dw=4 * H, ws=0), "dx dw ws"),
    look: (dict(ids=4 * R, table=2 * V * H, out=ROWS, ws=16), "out ws"),
    grad: (dict(ids=4 * R, dout=ROWS, dw=4 * V * H, ws=0), "dw ws"),
    clip: (dict(a=ROWS, b=28, oa=2 * ROWS, ob=14, norm=4, ws=0), "oa ob norm ws"),
    norm_alone: (dict(a=ROWS, b=28, norm=4, ws=0), "norm ws"),
}
ALIGN = dict(ws=256, ids=4, mask=1, scale=4, norm=4, a=2, b=4, oa=4, ob=2)
PAIRS = [(c, x, y) for c, (bufs, written) in CALLS.items() for x, y in itertools.permutations(bufs, 2)
         if x in written.split() or y in written.split()]


def workspace(lib, call):
    if call is bwd:
        return lib.eas_rmsnorm_bwd_workspace_size(R, H)
    return lib.eas_embed_bwd_workspace_size(R, H, V) if call is grad else lib.eas_clip_grad_norm_workspace_size(2)


@pytest.mark.parametrize("call,x,y", PAIRS, ids=lambda v: v if isinstance(v, str) else v.__name__)
def test_overlaps_are_refused(libeas, call, x, y):
    bufs = CALLS[call][0]
    p = {name: (i + 1) << 24 for i, name in enumerate(bufs)}
    n = bufs[x] or workspace(libeas, call)
    # y starts in x's last bytes, and in x's first ones
    a = ALIGN.get(y, 16)
    at = {p[x] + (n - 1) // a * a}
    if n > a:
        at.add(p[x] + a)
    for q in at:
        assert call(libeas, {**p, y: q}) == _lib.EAS_ERR_INVALID_ARG
        assert b"overlaps" in libeas.eas_last_error()


@pytest.mark.parametrize("call,x,y", [(fwd, "w", "s"), (fwd, "x", "y"), (bwd, "dy", "dx"), (bwd, "s", "dx"),
                                      (grad, "dout", "dw"), (look, "table", "out"), (clip, "b", "oa")],
                         ids=lambda v: v if isinstance(v, str) else v.__name__)
def test_only_the_named_buffers_may_be_replaced(libeas, call, x, y):
    p = {name: (i + 1) << 24 for i, name in enumerate(CALLS[call][0])}
    assert call(libeas, {**p, y: p[x]}) == _lib.EAS_ERR_INVALID_ARG
    assert b"overlaps" in libeas.eas_last_error()
