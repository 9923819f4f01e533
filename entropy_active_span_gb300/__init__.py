"""GB300 (sm_103a) block-sparse fused LM-head.

Python binding of the C ABI in include/eas.h.  Every function here only
checks and marshals arguments (device pointers, sizes, the current CUDA
stream) and calls the library; all arithmetic runs in the library's CUDA
kernels.  PyTorch provides device memory and streams.

    spans, num_spans = build_active_spans(mask, max_gap=128)
    logprob, entropy, lse = lmhead_fwd(hidden, weight, targets, mask, spans, num_spans)
    dhidden, dweight = lmhead_bwd(g_logprob, g_entropy, hidden, weight, targets, mask,
                                  spans, num_spans, lse, entropy)

Around the LM head: the embedding lookup and its gradient, the residual RMS
norm (bf16 or fp32, with e4m3 codes for lmhead_fwd_fp8) and its backward, and
the clipping of all gradients by their global norm.

    x = embed_fwd(ids, table, scale)
    y, y_e4m3, y_scale, s = rmsnorm_fwd(x, norm_weight, eps, residual=r, mask=mask,
                                        want_e4m3=True)
    ds, dnorm_weight = rmsnorm_bwd(dhidden, s, norm_weight, eps, mask=mask)
    embed_bwd(ids, ds, V, scale, accumulate=True, dweight=dweight)   # tied weights
    norm = clip_grad_norm([dweight, dnorm_weight], max_norm)
"""
from __future__ import annotations

import ctypes
from array import array

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import (EAS_BF16, EAS_DEFAULT_VOCAB_CHUNK, EAS_E4M3, EAS_FP32, EAS_MAX_TOKENS, EAS_MAX_TOP,
                   EAS_REUSE_FWD_ROWS, EAS_ROWS_ACTIVE, EAS_ROWS_SPAN, EasError)

__all__ = [
    "build_active_spans", "lmhead_fwd", "lmhead_bwd", "lmhead_workspace_size",
    "spans_workspace_size", "read_device_status", "workspace", "EasError",
    "EAS_ROWS_ACTIVE", "EAS_ROWS_SPAN", "EAS_REUSE_FWD_ROWS", "EAS_DEFAULT_VOCAB_CHUNK",
    "FusedLMHeadLogprob",
    "fused_logprob_entropy", "trace_enable", "trace_read", "lmhead_fwd_shard",
    "lmhead_combine_shards", "lmhead_bwd_shard", "cp_local_layout", "quantize_rows_e4m3",
    "lmhead_fwd_fp8", "lmhead_bwd_fp8", "lmhead_bwd_fp8_workspace_size",
    "rmsnorm_fwd", "rmsnorm_bwd", "rmsnorm_bwd_workspace_size", "FusedRMSNorm", "fused_rmsnorm",
    "embed_fwd", "embed_bwd", "embed_bwd_workspace_size", "FusedEmbedding", "fused_embedding",
    "clip_grad_norm", "clip_grad_norm_workspace_size",
    "EAS_MAX_TOKENS", "EAS_MAX_TOP", "token_logprobs_fwd", "token_logprobs_bwd",
    "FusedTokenLogprobs", "fused_token_logprobs",
    "NEWTON_SCHULZ", "orthogonalize", "muon_update", "orthogonalize_workspace_size",
]


def _ptr(t):
    return None if t is None else ctypes_ptr(t)


def ctypes_ptr(t: torch.Tensor) -> int:
    return t.data_ptr()


# The handle alone where torch has the call for it: a Stream object costs 2 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return EAS_BF16
    if dt == torch.float32:
        return EAS_FP32
    if dt in (torch.uint8, torch.float8_e4m3fn):
        return EAS_E4M3
    raise TypeError(f"hidden/weight must be bfloat16, float32 or e4m3, got {dt}")


def _as_codes(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, device) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def spans_workspace_size(T: int) -> int:
    return int(_lib.load().eas_spans_workspace_size(T))


def lmhead_workspace_size(T: int, H: int, V: int, dtype: torch.dtype,
                          vocab_chunk: int = 0) -> int:
    return int(_lib.load().eas_lmhead_workspace_size(T, H, V, _dtype_code(dtype), vocab_chunk))


def workspace(nbytes: int, device) -> torch.Tensor:
    """A device buffer usable as workspace (torch's allocator aligns to 512 B)."""
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def build_active_spans(mask: torch.Tensor, max_gap: int = 128, cap: int | None = None,
                       spans: torch.Tensor | None = None, num_spans: torch.Tensor | None = None,
                       ws: torch.Tensor | None = None):
    """Ordered active spans of a uint8 loss mask, built on the device.

    Returns (spans int32 [cap, 2], num_spans int32 [1]); only the first
    num_spans rows are meaningful.  cap defaults to the worst case (T+1)//2."""
    dev = mask.device
    _need(mask, "mask", torch.uint8, dev)
    T = mask.numel()
    if cap is None:
        cap = max(1, (T + 1) // 2)
    if spans is None:
        spans = torch.empty((cap, 2), dtype=torch.int32, device=dev)
    if num_spans is None:
        num_spans = torch.empty(1, dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(spans_workspace_size(T), dev)
    _need(spans, "spans", torch.int32, dev)
    _need(num_spans, "num_spans", torch.int32, dev)
    _lib.check(_lib.load().eas_build_active_spans(
        _ptr(mask), T, int(max_gap), _ptr(spans), int(spans.shape[0]), _ptr(num_spans),
        _ptr(ws), ws.numel(), _stream(dev)))
    return spans, num_spans


def cp_local_layout(mask, seg_offsets, cp_size: int, cp_rank: int, ws=None):
    """(local_mask uint8 [T/cp], local_to_global int32 [T/cp]) of one CP rank
    under the load-balanced split of every packed segment into 2*cp chunks."""
    dev = mask.device
    _need(mask, "mask", torch.uint8, dev)
    _need(seg_offsets, "seg_offsets", torch.int32, dev)
    T = mask.numel()
    n_local = T // cp_size
    local_mask = torch.empty(n_local, dtype=torch.uint8, device=dev)
    l2g = torch.empty(n_local, dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(64, dev)
    _lib.check(_lib.load().eas_cp_local_layout(
        _ptr(mask), _ptr(seg_offsets), int(seg_offsets.numel() - 1), T, int(cp_size),
        int(cp_rank), _ptr(local_mask), _ptr(l2g), _ptr(ws), ws.numel(), _stream(dev)))
    return local_mask, l2g


def lmhead_fwd(hidden, weight, targets, mask, spans, num_spans, flags: int = EAS_ROWS_ACTIVE,
               ws=None, out=None, want_lse: bool = True):
    """Target logprob, entropy and lse of the active rows.  Returns (logprob, entropy, lse).

    With want_lse=False (forward-only scoring) lse is neither computed into
    memory nor returned (None)."""
    dev = hidden.device
    dt = hidden.dtype
    code = _dtype_code(dt)
    T, H = hidden.shape
    V = weight.shape[0]
    _need(hidden, "hidden", dt, dev)
    _need(weight, "weight", dt, dev)
    if weight.shape[1] != H:
        raise ValueError("weight must be [V, H]")
    _need(targets, "targets", torch.int32, dev)
    _need(mask, "mask", torch.uint8, dev)
    _need(spans, "spans", torch.int32, dev)
    _need(num_spans, "num_spans", torch.int32, dev)
    if targets.numel() != T or mask.numel() != T:
        raise ValueError("targets and mask must have T entries")
    if out is None:
        out = tuple(torch.empty(T, dtype=torch.float32, device=dev) for _ in range(3))
    if ws is None:
        ws = workspace(lmhead_workspace_size(T, H, V, dt), dev)
    logprob, entropy, lse = out
    if not want_lse:
        lse = None
    _lib.check(_lib.load().eas_lmhead_fwd(
        _ptr(hidden), _ptr(weight), _ptr(targets), _ptr(mask), _ptr(spans), _ptr(num_spans),
        int(spans.shape[0]), T, H, V, code, int(flags), _ptr(logprob), _ptr(entropy), _ptr(lse),
        _ptr(ws), ws.numel(), _stream(dev)))
    return logprob, entropy, lse


def lmhead_bwd(g_logprob, g_entropy, hidden, weight, targets, mask, spans, num_spans, lse,
               entropy, flags: int = EAS_ROWS_ACTIVE, vocab_chunk: int = 0, ws=None,
               dhidden=None, dweight=None):
    """dHidden (hidden's dtype) and dW (fp32) of sum_active g_lp logp + g_H H."""
    dev = hidden.device
    dt = hidden.dtype
    code = _dtype_code(dt)
    T, H = hidden.shape
    V = weight.shape[0]
    for t, n in ((g_logprob, "g_logprob"), (g_entropy, "g_entropy"), (lse, "lse"),
                 (entropy, "entropy")):
        _need(t, n, torch.float32, dev)
        if t.numel() != T:
            raise ValueError(f"{n} must have T entries")
    _need(hidden, "hidden", dt, dev)
    _need(weight, "weight", dt, dev)
    _need(targets, "targets", torch.int32, dev)
    _need(mask, "mask", torch.uint8, dev)
    _need(spans, "spans", torch.int32, dev)
    _need(num_spans, "num_spans", torch.int32, dev)
    if dhidden is None:
        dhidden = torch.empty((T, H), dtype=dt, device=dev)
    if dweight is None:
        dweight = torch.empty((V, H), dtype=torch.float32, device=dev)
    _need(dhidden, "dhidden", dt, dev)
    _need(dweight, "dweight", torch.float32, dev)
    if ws is None:
        ws = workspace(lmhead_workspace_size(T, H, V, dt, vocab_chunk), dev)
    _lib.check(_lib.load().eas_lmhead_bwd(
        _ptr(g_logprob), _ptr(g_entropy), _ptr(hidden), _ptr(weight), _ptr(targets), _ptr(mask),
        _ptr(spans), _ptr(num_spans), int(spans.shape[0]), _ptr(lse), _ptr(entropy),
        T, H, V, code, int(flags), int(vocab_chunk), _ptr(dhidden), _ptr(dweight),
        _ptr(ws), ws.numel(), _stream(dev)))
    return dhidden, dweight


def quantize_rows_e4m3(x: torch.Tensor, out=None, scale=None):
    """Per-row e4m3 quantisation of a bf16/fp32 [R, H] tensor on the device.
    Returns (codes uint8 [R, H], scale fp32 [R])."""
    dev = x.device
    code = _dtype_code(x.dtype)
    if code == EAS_E4M3:
        raise TypeError("x must be bfloat16 or float32")
    _need(x, "x", x.dtype, dev)
    R, H = x.shape
    if out is None:
        out = torch.empty((R, H), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = torch.empty(R, dtype=torch.float32, device=dev)
    _lib.check(_lib.load().eas_quantize_rows_e4m3(_ptr(x), code, R, H, _ptr(out), _ptr(scale),
                                                  _stream(dev)))
    return out, scale


def lmhead_fwd_fp8(hidden_e4m3, hidden_scale, weight_e4m3, weight_scale, targets, mask, spans,
                   num_spans, flags: int = EAS_ROWS_ACTIVE, ws=None, out=None,
                   want_lse: bool = True):
    """Forward with e4m3 operands and per-row scales (forward-only scoring)."""
    h8, w8 = _as_codes(hidden_e4m3), _as_codes(weight_e4m3)
    dev = h8.device
    T, H = h8.shape
    V = w8.shape[0]
    for t, n, d in ((h8, "hidden_e4m3", torch.uint8), (w8, "weight_e4m3", torch.uint8),
                    (hidden_scale, "hidden_scale", torch.float32),
                    (weight_scale, "weight_scale", torch.float32),
                    (targets, "targets", torch.int32), (mask, "mask", torch.uint8),
                    (spans, "spans", torch.int32), (num_spans, "num_spans", torch.int32)):
        _need(t, n, d, dev)
    if out is None:
        out = tuple(torch.empty(T, dtype=torch.float32, device=dev) for _ in range(3))
    lp, ent, lse = out
    if not want_lse:
        lse = None
    if ws is None:
        ws = workspace(lmhead_workspace_size(T, H, V, torch.uint8), dev)
    _lib.check(_lib.load().eas_lmhead_fwd_fp8(
        _ptr(h8), _ptr(hidden_scale), _ptr(w8), _ptr(weight_scale), _ptr(targets), _ptr(mask),
        _ptr(spans), _ptr(num_spans), int(spans.shape[0]), T, H, V, int(flags), _ptr(lp),
        _ptr(ent), _ptr(lse), _ptr(ws), ws.numel(), _stream(dev)))
    return lp, ent, lse


def lmhead_bwd_fp8_workspace_size(T: int, H: int, V: int, vocab_chunk: int = 0) -> int:
    return int(_lib.load().eas_lmhead_bwd_fp8_workspace_size(T, H, V, vocab_chunk))


def lmhead_bwd_fp8(g_logprob, g_entropy, hidden, weight, hidden_e4m3, hidden_scale, weight_e4m3,
                   weight_scale, targets, mask, spans, num_spans, lse, entropy,
                   flags: int = EAS_ROWS_ACTIVE, vocab_chunk: int = 0, ws=None, dhidden=None,
                   dweight=None):
    """Backward of the e4m3 forward: d-logits of the e4m3 logits, projected
    with the bf16 operands.  Returns (dHidden bf16, dW fp32)."""
    dev = hidden.device
    T, H = hidden.shape
    V = weight.shape[0]
    h8, w8 = _as_codes(hidden_e4m3), _as_codes(weight_e4m3)
    for t, n, d in ((g_logprob, "g_logprob", torch.float32), (g_entropy, "g_entropy", torch.float32),
                    (lse, "lse", torch.float32), (entropy, "entropy", torch.float32),
                    (hidden, "hidden", torch.bfloat16), (weight, "weight", torch.bfloat16),
                    (h8, "hidden_e4m3", torch.uint8), (w8, "weight_e4m3", torch.uint8),
                    (hidden_scale, "hidden_scale", torch.float32),
                    (weight_scale, "weight_scale", torch.float32),
                    (targets, "targets", torch.int32), (mask, "mask", torch.uint8),
                    (spans, "spans", torch.int32), (num_spans, "num_spans", torch.int32)):
        _need(t, n, d, dev)
    if h8.shape != (T, H) or w8.shape != (V, H):
        raise ValueError("the e4m3 operands must have the shapes of hidden and weight")
    if dhidden is None:
        dhidden = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if dweight is None:
        dweight = torch.empty((V, H), dtype=torch.float32, device=dev)
    _need(dhidden, "dhidden", torch.bfloat16, dev)
    _need(dweight, "dweight", torch.float32, dev)
    if ws is None:
        ws = workspace(lmhead_bwd_fp8_workspace_size(T, H, V, vocab_chunk), dev)
    _lib.check(_lib.load().eas_lmhead_bwd_fp8(
        _ptr(g_logprob), _ptr(g_entropy), _ptr(hidden), _ptr(weight), _ptr(h8), _ptr(hidden_scale),
        _ptr(w8), _ptr(weight_scale), _ptr(targets), _ptr(mask), _ptr(spans), _ptr(num_spans),
        int(spans.shape[0]), _ptr(lse), _ptr(entropy), T, H, V, int(flags), int(vocab_chunk),
        _ptr(dhidden), _ptr(dweight), _ptr(ws), ws.numel(), _stream(dev)))
    return dhidden, dweight


def lmhead_fwd_shard(hidden, weight_shard, v_lo: int, targets, mask, spans, num_spans,
                     flags: int = EAS_ROWS_ACTIVE, ws=None, stats=None):
    """Per-token (M, S, U, z) statistics of one vocabulary shard ([T, 4] fp32)."""
    dev = hidden.device
    dt = hidden.dtype
    T, H = hidden.shape
    Vs = weight_shard.shape[0]
    for t, n, d in ((hidden, "hidden", dt), (weight_shard, "weight_shard", dt),
                    (targets, "targets", torch.int32), (mask, "mask", torch.uint8),
                    (spans, "spans", torch.int32), (num_spans, "num_spans", torch.int32)):
        _need(t, n, d, dev)
    if stats is None:
        stats = torch.empty((T, 4), dtype=torch.float32, device=dev)
    _need(stats, "stats", torch.float32, dev)
    if ws is None:
        ws = workspace(lmhead_workspace_size(T, H, Vs, dt), dev)
    _lib.check(_lib.load().eas_lmhead_fwd_shard(
        _ptr(hidden), _ptr(weight_shard), int(v_lo), _ptr(targets), _ptr(mask), _ptr(spans),
        _ptr(num_spans), int(spans.shape[0]), T, H, Vs, _dtype_code(dt), int(flags),
        _ptr(stats), _ptr(ws), ws.numel(), _stream(dev)))
    return stats


def lmhead_combine_shards(stats, mask, out=None, want_lse: bool = True):
    """Merges [n_shards, T, 4] shard statistics into (logprob, entropy, lse)."""
    dev = stats.device
    n, T = int(stats.shape[0]), int(stats.shape[1])
    _need(stats, "stats", torch.float32, dev)
    _need(mask, "mask", torch.uint8, dev)
    if out is None:
        out = tuple(torch.empty(T, dtype=torch.float32, device=dev) for _ in range(3))
    lp, ent, lse = out
    if not want_lse:
        lse = None
    _lib.check(_lib.load().eas_lmhead_combine_shards(_ptr(stats), n, T, _ptr(mask), _ptr(lp),
                                                     _ptr(ent), _ptr(lse), _stream(dev)))
    return lp, ent, lse


def lmhead_bwd_shard(g_logprob, g_entropy, hidden, weight_shard, v_lo: int, targets, mask, spans,
                     num_spans, lse, entropy, flags: int = EAS_ROWS_ACTIVE, vocab_chunk: int = 0,
                     ws=None, dhidden_partial=None, dweight_shard=None):
    """This shard's dW rows and partial dHidden (the partials sum to dHidden)."""
    dev = hidden.device
    dt = hidden.dtype
    T, H = hidden.shape
    Vs = weight_shard.shape[0]
    for t, n in ((g_logprob, "g_logprob"), (g_entropy, "g_entropy"), (lse, "lse"),
                 (entropy, "entropy")):
        _need(t, n, torch.float32, dev)
    for t, n, d in ((hidden, "hidden", dt), (weight_shard, "weight_shard", dt),
                    (targets, "targets", torch.int32), (mask, "mask", torch.uint8),
                    (spans, "spans", torch.int32), (num_spans, "num_spans", torch.int32)):
        _need(t, n, d, dev)
    if dhidden_partial is None:
        dhidden_partial = torch.empty((T, H), dtype=dt, device=dev)
    if dweight_shard is None:
        dweight_shard = torch.empty((Vs, H), dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(lmhead_workspace_size(T, H, Vs, dt, vocab_chunk), dev)
    _lib.check(_lib.load().eas_lmhead_bwd_shard(
        _ptr(g_logprob), _ptr(g_entropy), _ptr(hidden), _ptr(weight_shard), int(v_lo),
        _ptr(targets), _ptr(mask), _ptr(spans), _ptr(num_spans), int(spans.shape[0]), _ptr(lse),
        _ptr(entropy), T, H, Vs, _dtype_code(dt), int(flags), int(vocab_chunk),
        _ptr(dhidden_partial), _ptr(dweight_shard), _ptr(ws), ws.numel(), _stream(dev)))
    return dhidden_partial, dweight_shard


def read_device_status(ws: torch.Tensor) -> int:
    """Waits for the current stream and returns the status word in `ws` (0 = OK)."""
    st = _lib.load().eas_read_device_status(_ptr(ws), _stream(ws.device))
    return int(st)


def trace_enable(on: bool = True) -> None:
    """Start (clearing old records) or stop per-kernel event timing in the library."""
    _lib.load().eas_trace_enable(1 if on else 0)


def trace_read() -> list[tuple[str, float]]:
    """(kernel name, milliseconds) of every launch recorded since trace_enable(True)."""
    lib = _lib.load()
    n = lib.eas_trace_read(None, None, 0)
    kinds = (ctypes.c_int32 * max(n, 1))()
    ms = (ctypes.c_float * max(n, 1))()
    n = lib.eas_trace_read(kinds, ms, n)
    return [(lib.eas_kernel_name(kinds[i]).decode(), float(ms[i])) for i in range(n)]


class FusedLMHeadLogprob(torch.autograd.Function):
    """Autograd wrapper: (hidden, weight) -> (logprob, entropy) of the active rows.

    The backward feeds the upstream gradients of logprob and entropy to
    lmhead_bwd; weight's gradient is returned in weight's dtype."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, mask, spans, num_spans, flags, vocab_chunk):
        logprob, entropy, lse = lmhead_fwd(hidden, weight, targets, mask, spans, num_spans, flags)
        ctx.save_for_backward(hidden, weight, targets, mask, spans, num_spans, lse, entropy)
        ctx.flags, ctx.vocab_chunk = flags, vocab_chunk
        return logprob, entropy

    @staticmethod
    def backward(ctx, g_logprob, g_entropy):
        hidden, weight, targets, mask, spans, num_spans, lse, entropy = ctx.saved_tensors
        if g_logprob is None:
            g_logprob = torch.zeros_like(lse)
        if g_entropy is None:
            g_entropy = torch.zeros_like(lse)
        dh, dw = lmhead_bwd(g_logprob.contiguous().float(), g_entropy.contiguous().float(),
                            hidden, weight, targets, mask, spans, num_spans, lse, entropy,
                            ctx.flags, ctx.vocab_chunk)
        return dh, dw.to(weight.dtype), None, None, None, None, None, None


def fused_logprob_entropy(hidden, weight, targets, mask, spans=None, num_spans=None,
                          max_gap: int = 128, flags: int = EAS_ROWS_ACTIVE, vocab_chunk: int = 0):
    """Differentiable (logprob, entropy) of the active rows; builds the spans
    from the mask on the device when they are not given.  Under
    torch.no_grad() (or when neither input needs a gradient) it runs the
    forward alone and keeps no lse."""
    if spans is None or num_spans is None:
        spans, num_spans = build_active_spans(mask, max_gap)
    if not (torch.is_grad_enabled() and (hidden.requires_grad or weight.requires_grad)):
        lp, ent, _ = lmhead_fwd(hidden, weight, targets, mask, spans, num_spans, flags,
                                want_lse=False)
        return lp, ent
    return FusedLMHeadLogprob.apply(hidden, weight, targets, mask, spans, num_spans, flags,
                                    vocab_chunk)


# ------------------------------------------------- operators around the LM head

_ROW_CODES = {torch.bfloat16: EAS_BF16, torch.float32: EAS_FP32}


def _row_code(t: torch.Tensor, name: str) -> int:
    """dtype code of a row operator's tensor; refuses what no kernel can read."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device, got {t.device}")
    code = _ROW_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def _row_codes(ts, name: str) -> array:
    """_row_code of each tensor of a list (of the first one's device: the caller
    checks that the others are on it)."""
    try:
        codes = array("i", [_ROW_CODES[t.dtype] for t in ts])
        if ts[0].is_cuda:
            return codes
    except (AttributeError, KeyError):
        pass
    return array("i", [_row_code(t, name) for t in ts])


def _need_shape(t: torch.Tensor, name: str, dtype: torch.dtype, device, shape) -> None:
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == device and t.is_contiguous()):
        return
    _need(t, name, dtype, device)
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _ws_args(ws, device) -> tuple[int, int]:
    """Address and bytes of a workspace; refuses one that the kernels cannot write."""
    if not isinstance(ws, torch.Tensor):
        raise TypeError("ws must be a tensor")
    if ws.device != device:
        raise ValueError(f"ws is on {ws.device}, expected {device}")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def rmsnorm_fwd(x, weight, eps: float = 1e-6, residual=None, mask=None, want_y: bool = True,
                want_e4m3: bool = False, want_sum: bool = True, out=None):
    """RMS norm of x + residual ([R, H], bf16 or fp32) times weight [H].

    Returns (y, y_e4m3, y_scale, s): y in x's dtype (None without want_y), its
    e4m3 codes and row scales as lmhead_fwd_fp8 takes them (None without
    want_e4m3), and s = x + residual, which rmsnorm_bwd takes (x itself without
    a residual; None without want_sum).  Rows whose mask byte is 0 get y = 0,
    zero codes and scale 1.  out: buffers for the four, None where one is to be
    allocated; s may be x or residual itself."""
    code = _row_code(x, "x")
    dev, dt, shape = x.device, x.dtype, x.shape
    if len(shape) != 2:
        raise ValueError("x must be [R, H]")
    R, H = shape
    _need_shape(x, "x", dt, dev, shape)
    _need_shape(weight, "weight", dt, dev, (H,))
    r = m = yp = qp = sp = scp = None
    if residual is not None:
        _need_shape(residual, "residual", dt, dev, shape)
        r = residual.data_ptr()
    if mask is not None:
        _need_shape(mask, "mask", torch.uint8, dev, (R,))
        m = mask.data_ptr()
    y, q, scale, s = out if out is not None else (None, None, None, None)
    if want_y:
        if y is None:
            y = torch.empty_like(x)
        else:
            _need_shape(y, "y", dt, dev, shape)
        yp = y.data_ptr()
    else:
        y = None
    if want_e4m3:
        if q is None:
            q = torch.empty(shape, dtype=torch.uint8, device=dev)
        else:
            q = _as_codes(q)
            _need_shape(q, "y_e4m3", torch.uint8, dev, shape)
        if scale is None:
            scale = torch.empty(R, dtype=torch.float32, device=dev)
        else:
            _need_shape(scale, "y_scale", torch.float32, dev, (R,))
        qp, scp = q.data_ptr(), scale.data_ptr()
    else:
        q = scale = None
    if not want_sum:
        s = None
    elif residual is None:
        s = x
    else:
        if s is None:
            s = torch.empty_like(x)
        else:
            _need_shape(s, "s", dt, dev, shape)
        sp = s.data_ptr()
    _lib.check(_lib.load().eas_rmsnorm_fwd(x.data_ptr(), r, weight.data_ptr(), m, R, H, code, eps,
                                           sp, yp, qp, scp, _stream(dev)))
    return y, q, scale, s


def rmsnorm_bwd_workspace_size(R: int, H: int) -> int:
    return int(_lib.load().eas_rmsnorm_bwd_workspace_size(R, H))


def rmsnorm_bwd(dy, s, weight, eps: float = 1e-6, ds=None, mask=None, ws=None, dx=None,
                dweight=None):
    """Gradients of rmsnorm_fwd's y: (dx in s's dtype, dweight fp32).

    s is the forward's sum; dx is the gradient of x and of the residual alike.
    ds, the gradient arriving at s from elsewhere, is added to dx (and may be
    the dx buffer).  Inactive rows' dx is ds or 0."""
    code = _row_code(s, "s")
    dev, dt = s.device, s.dtype
    if s.dim() != 2:
        raise ValueError("s must be [R, H]")
    R, H = s.shape
    _need(s, "s", dt, dev)
    _need_shape(dy, "dy", dt, dev, s.shape)
    _need_shape(weight, "weight", dt, dev, (H,))
    if ds is not None:
        _need_shape(ds, "ds", dt, dev, s.shape)
    if mask is not None:
        _need_shape(mask, "mask", torch.uint8, dev, (R,))
    if dx is None:
        dx = torch.empty_like(s)
    else:
        _need_shape(dx, "dx", dt, dev, s.shape)
    if dweight is None:
        dweight = torch.empty(H, dtype=torch.float32, device=dev)
    else:
        _need_shape(dweight, "dweight", torch.float32, dev, (H,))
    if ws is None:
        ws = workspace(rmsnorm_bwd_workspace_size(R, H), dev)
    _lib.check(_lib.load().eas_rmsnorm_bwd(
        _ptr(dy), _ptr(s), _ptr(weight), _ptr(ds), _ptr(mask), R, H, code, eps, _ptr(dx),
        _ptr(dweight), *_ws_args(ws, dev), _stream(dev)))
    return dx, dweight


def embed_fwd(ids, table, scale: float = 1.0, ws=None, out=None):
    """scale * table[ids] ([T, H] in table's dtype); id -1 is padding (a zero row).

    Other ids outside the table give zero rows and, where ws (16 bytes or
    more) is passed, EAS_ERR_INVALID_ARG in its status word."""
    code = _row_code(table, "table")
    dev, dt = table.device, table.dtype
    if table.dim() != 2:
        raise ValueError("table must be [V, H]")
    V, H = table.shape
    _need(table, "table", dt, dev)
    _need(ids, "ids", torch.int32, dev)
    T = ids.numel()
    if out is None:
        out = torch.empty((T, H), dtype=dt, device=dev)
    else:
        _need_shape(out, "out", dt, dev, (T, H))
    _lib.check(_lib.load().eas_embed_fwd(
        _ptr(ids), _ptr(table), T, H, V, code, scale, _ptr(out),
        *((None, 0) if ws is None else _ws_args(ws, dev)), _stream(dev)))
    return out


def embed_bwd_workspace_size(T: int, H: int, V: int) -> int:
    return int(_lib.load().eas_embed_bwd_workspace_size(T, H, V))


def embed_bwd(ids, dout, V: int, scale: float = 1.0, accumulate: bool = False, ws=None,
              dweight=None):
    """Gradient of embed_fwd's table: fp32 [V, H], summed in a fixed order.

    With accumulate the sums are added to dweight (tied weights: lmhead_bwd's),
    else every row of it is written."""
    code = _row_code(dout, "dout")
    dev, dt = dout.device, dout.dtype
    if dout.dim() != 2:
        raise ValueError("dout must be [T, H]")
    T, H = dout.shape
    _need(dout, "dout", dt, dev)
    _need(ids, "ids", torch.int32, dev)
    if ids.numel() != T:
        raise ValueError("ids must have T entries")
    if dweight is None:
        if accumulate:
            raise ValueError("accumulate needs dweight")
        dweight = torch.empty((V, H), dtype=torch.float32, device=dev)
    else:
        _need_shape(dweight, "dweight", torch.float32, dev, (V, H))
    if ws is None:
        ws = workspace(embed_bwd_workspace_size(T, H, V), dev)
    _lib.check(_lib.load().eas_embed_bwd(
        _ptr(ids), _ptr(dout), T, H, V, code, scale, 1 if accumulate else 0, _ptr(dweight),
        *_ws_args(ws, dev), _stream(dev)))
    return dweight


def clip_grad_norm_workspace_size(n: int) -> int:
    return int(_lib.load().eas_clip_grad_norm_workspace_size(n))


def clip_grad_norm(grads, max_norm: float | None, out=None, ws=None, norm=None):
    """Scales gradients by min(1, max_norm / (norm + 1e-6)), norm being the
    2-norm over all of them, and returns norm (fp32 [1], on the device).

    grads: contiguous bf16 or fp32 tensors.  out: None scales in place; else one
    tensor for each gradient, of its size, bf16 or fp32 (an fp32 gradient
    clipped into the bf16 one that an optimiser reads).  max_norm None computes
    the norm alone.  Where the norm is not finite nothing is scaled."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    n = len(grads)
    if len(outs) != n:
        raise ValueError("out must have one tensor for each gradient")
    if n == 0:
        raise ValueError("no gradients")
    # maps over the methods themselves: a list has hundreds of tensors, and what
    # the host does for each is the whole time of a small call
    T = torch.Tensor
    codes = _row_codes(grads, "grads")
    dev, index = grads[0].device, grads[0].get_device()
    if not (all(map(T.is_contiguous, grads)) and set(map(T.get_device, grads)) == {index}):
        raise ValueError(f"gradients must be contiguous and on one device ({dev})")
    ptrs, numels = array("Q", map(T.data_ptr, grads)), array("q", map(T.numel, grads))
    out_codes, out_ptrs = codes, ptrs
    if out is not None:
        out_codes = _row_codes(outs, "out")
        if not (all(map(T.is_contiguous, outs)) and set(map(T.get_device, outs)) == {index}
                and numels == array("q", map(T.numel, outs))):
            raise ValueError("out must be contiguous and have the gradients' sizes and device")
        out_ptrs = array("Q", map(T.data_ptr, outs))
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=dev)
    else:
        _need_shape(norm, "norm", torch.float32, dev, (1,))
    if ws is None:
        ws = workspace(clip_grad_norm_workspace_size(n), dev)
    clip = max_norm is not None
    _lib.check(_lib.load().eas_clip_grad_norm(
        ptrs.buffer_info()[0], out_ptrs.buffer_info()[0] if clip else None,
        numels.buffer_info()[0], codes.buffer_info()[0], out_codes.buffer_info()[0], n,
        max_norm if clip else 0.0, norm.data_ptr(), *_ws_args(ws, dev), _stream(dev)))
    return norm


def _rows_of(t: torch.Tensor, name: str) -> int:
    """Row pitch of a matrix whose rows are dense (a slice of wider rows, say)."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be [N, V]")
    N, V = t.shape
    if V > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have dense rows")
    if N <= 1:
        return V
    if t.stride(0) < V:
        raise ValueError(f"{name} must not have rows that overlap")
    return t.stride(0)


def _token_list(tokens, N: int, device) -> int:
    """Tokens a row of a [N] or [N, M] list."""
    if tokens is None:
        return 0
    _need(tokens, "tokens", torch.int32, device)
    if tokens.dim() not in (1, 2) or tokens.shape[0] != N:
        raise ValueError(f"tokens must be [N] or [N, M] with N = {N}, got {tuple(tokens.shape)}")
    return 1 if tokens.dim() == 1 else tokens.shape[1]


def token_logprobs_fwd(logits, tokens=None, top_k: int = 0, scale: float = 1.0, mask=None, ws=None,
                       out=None):
    """Scores of existing logits ([N, V], bf16 or fp32, rows dense but any pitch).

    Returns (logprob, entropy, lse, top_logprob, top_ids) of softmax(scale * logits):
    the log probabilities of tokens ([N] or [N, M] int32; -1: none, 0), the entropy
    and log-sum-exp of each row, and the top_k likeliest tokens of each row with
    their log probabilities, ties by ascending id.  logprob is None without tokens,
    the last two without top_k.  Rows whose mask byte is 0 are not read and get
    zeros (top_ids -1).  Tokens outside the vocabulary get 0 and, where ws (16
    bytes or more) is passed, EAS_ERR_INVALID_ARG in its status word.  out: buffers
    for the five, None where one is to be allocated."""
    code = _row_code(logits, "logits")
    dev = logits.device
    ld = _rows_of(logits, "logits")
    N, V = logits.shape
    M = _token_list(tokens, N, dev)
    if mask is not None:
        _need_shape(mask, "mask", torch.uint8, dev, (N,))
    wanted = [(None if tokens is None else tokens.shape, torch.float32, "logprob"),
              ((N,), torch.float32, "entropy"), ((N,), torch.float32, "lse"),
              ((N, top_k) if top_k else None, torch.float32, "top_logprob"),
              ((N, top_k) if top_k else None, torch.int32, "top_ids")]
    res = list(out) if out is not None else [None] * 5
    for i, (shape, dt, name) in enumerate(wanted):
        if shape is None:
            res[i] = None
        elif res[i] is None:
            res[i] = torch.empty(shape, dtype=dt, device=dev)
        else:
            _need_shape(res[i], name, dt, dev, shape)
    lp, ent, lse, top, ids = res
    _lib.check(_lib.load().eas_token_logprobs_fwd(
        _ptr(logits), ld, _ptr(tokens), _ptr(mask), N, V, M, top_k, code, scale, _ptr(lp),
        _ptr(ent), _ptr(lse), _ptr(top), _ptr(ids),
        *((None, 0) if ws is None else _ws_args(ws, dev)), _stream(dev)))
    return lp, ent, lse, top, ids


def token_logprobs_bwd(g_logprob, g_entropy, logits, tokens, lse, entropy, scale: float = 1.0,
                       mask=None, ws=None, out=None):
    """Gradient of token_logprobs_fwd's logprob and entropy at the logits, in their dtype.

    g_logprob has the shape of tokens (both None: no given tokens), g_entropy is [N]
    or None.  lse and entropy are the forward's.  top_logprob's gradient is that of
    tokens: append top_ids to them.  out may be logits itself."""
    code = _row_code(logits, "logits")
    dev = logits.device
    ld = _rows_of(logits, "logits")
    N, V = logits.shape
    M = _token_list(tokens, N, dev)
    if (tokens is None) != (g_logprob is None):
        raise ValueError("tokens and g_logprob come together")
    if tokens is not None:
        _need_shape(g_logprob, "g_logprob", torch.float32, dev, tokens.shape)
    if g_entropy is not None:
        _need_shape(g_entropy, "g_entropy", torch.float32, dev, (N,))
    _need_shape(lse, "lse", torch.float32, dev, (N,))
    _need_shape(entropy, "entropy", torch.float32, dev, (N,))
    if mask is not None:
        _need_shape(mask, "mask", torch.uint8, dev, (N,))
    if out is None:
        out = torch.empty((N, V), dtype=logits.dtype, device=dev)
    elif not isinstance(out, torch.Tensor) or out.dtype != logits.dtype or out.device != dev:
        raise TypeError(f"out must be a {logits.dtype} tensor on {dev}")
    elif out.shape != logits.shape:
        raise ValueError(f"out must have shape {(N, V)}, got {tuple(out.shape)}")
    _lib.check(_lib.load().eas_token_logprobs_bwd(
        _ptr(g_logprob), _ptr(g_entropy), _ptr(logits), ld, _ptr(tokens), _ptr(mask), _ptr(lse),
        _ptr(entropy), N, V, M, code, scale, _ptr(out), _rows_of(out, "out"),
        *((None, 0) if ws is None else _ws_args(ws, dev)), _stream(dev)))
    return out


def _grad_rows(g: torch.Tensor) -> torch.Tensor:
    """An upstream gradient as the kernels read it: dense, on a 16-byte boundary
    (autograd hands over broadcast and offset views)."""
    g = g.contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


class FusedRMSNorm(torch.autograd.Function):
    """Autograd wrapper of rmsnorm_fwd / rmsnorm_bwd: (y, s, y_e4m3, y_scale).

    The codes and scales carry no gradient: the LM head's e4m3 backward
    projects with the unquantised rows."""

    @staticmethod
    def forward(ctx, x, residual, weight, mask, eps, want_e4m3):
        y, q, scale, s = rmsnorm_fwd(x, weight, eps, residual, mask, want_e4m3=want_e4m3)
        ctx.save_for_backward(s, weight, mask)
        ctx.eps, ctx.has_residual = eps, residual is not None
        ctx.set_materialize_grads(False)
        if want_e4m3:
            ctx.mark_non_differentiable(q, scale)
        return y, (s if residual is not None else None), q, scale

    @staticmethod
    @once_differentiable
    def backward(ctx, g_y, g_s, _q, _scale):
        s, weight, mask = ctx.saved_tensors
        if g_y is None:
            dx, dw = g_s, None
        else:
            ds = None if g_s is None else _grad_rows(g_s)
            dx, dw = rmsnorm_bwd(_grad_rows(g_y), s, weight, ctx.eps, ds, mask)
            dw = dw.to(weight.dtype)
        return dx, (dx if ctx.has_residual else None), dw, None, None, None


def fused_rmsnorm(x, weight, residual=None, eps: float = 1e-6, mask=None,
                  want_e4m3: bool = False):
    """Differentiable RMS norm of x (+ residual): (y, s, y_e4m3, y_scale), s being
    None without a residual, the codes and scales None without want_e4m3."""
    return FusedRMSNorm.apply(x, residual, weight, mask, eps, want_e4m3)


class FusedEmbedding(torch.autograd.Function):
    """Autograd wrapper of embed_fwd / embed_bwd; the table's gradient is
    returned in the table's dtype."""

    @staticmethod
    def forward(ctx, ids, table, scale):
        ctx.save_for_backward(ids)
        ctx.V, ctx.dtype, ctx.scale = table.shape[0], table.dtype, scale
        return embed_fwd(ids, table, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        ids, = ctx.saved_tensors
        return None, embed_bwd(ids, _grad_rows(g), ctx.V, ctx.scale).to(ctx.dtype), None


def fused_embedding(ids, table, scale: float = 1.0):
    """Differentiable scale * table[ids] ([T, H]); id -1 is padding."""
    return FusedEmbedding.apply(ids, table, scale)


class FusedTokenLogprobs(torch.autograd.Function):
    """Autograd wrapper of token_logprobs_fwd / token_logprobs_bwd: logits ->
    (logprob, entropy, top_logprob, top_ids).  top_logprob's gradient goes to the
    tokens that were the top ones."""

    @staticmethod
    def forward(ctx, logits, tokens, top_k, scale, mask):
        lp, ent, lse, top, ids = token_logprobs_fwd(logits, tokens, top_k, scale, mask)
        ctx.save_for_backward(logits, tokens, lse, ent, ids, mask)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        if ids is not None:
            ctx.mark_non_differentiable(ids)
        return lp, ent, top, ids

    @staticmethod
    @once_differentiable
    def backward(ctx, g_lp, g_ent, g_top, _ids):
        logits, tokens, lse, ent, ids, mask = ctx.saved_tensors
        given = [tuple(v if v.dim() == 2 else v[:, None] for v in (t, g.float()))
                 for t, g in ((tokens, g_lp), (ids, g_top)) if g is not None]
        t = g = None
        if given:
            t, g = (torch.cat(p, 1) for p in zip(*given))
        if g_ent is not None:
            g_ent = g_ent.contiguous().float()
        return token_logprobs_bwd(g, g_ent, logits, t, lse, ent, ctx.scale, mask), None, None, None, None


def fused_token_logprobs(logits, tokens=None, top_k: int = 0, scale: float = 1.0, mask=None):
    """Differentiable (logprob, entropy, top_logprob, top_ids) of existing logits; see
    token_logprobs_fwd.  Without tokens logprob is None, without top_k the last two.
    tokens and top_k together are at most 128 a row."""
    if _token_list(tokens, logits.shape[0], logits.device) + top_k > EAS_MAX_TOKENS:
        raise ValueError(f"tokens and top_k together are at most {EAS_MAX_TOKENS} a row")
    return FusedTokenLogprobs.apply(logits, tokens, top_k, scale, mask)


# Coefficients (a, b, c) of a Newton-Schulz step that raise small singular values fast
# and bring all of them near 1 in about five steps: those of Keller Jordan's description
# of the Muon optimiser (2024).
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


def orthogonalize_workspace_size(L: int, rows: int, cols: int) -> int:
    return int(_lib.load().eas_orthogonalize_workspace_size(L, rows, cols))


def _coefficients(coeffs, steps: int) -> array:
    flat = list(coeffs)
    if flat and not hasattr(flat[0], "__len__"):
        flat = [flat] * steps
    if len(flat) != steps or any(len(c) != 3 for c in flat):
        raise ValueError("coeffs must be one (a, b, c) or one for each step")
    return array("f", [v for c in flat for v in c])


def _orthogonalize(grad, momentum, new_momentum, beta, nesterov, steps, coeffs, eps, scale, ws, out):
    code = _row_code(grad, "grad")
    dev, shape = grad.device, grad.shape
    if len(shape) not in (2, 3):
        raise ValueError("grad must be [rows, cols] or [L, rows, cols]")
    L, rows, cols = (1, *shape) if len(shape) == 2 else shape
    _need_shape(grad, "grad", grad.dtype, dev, shape)
    mom_code, mp, np_ = code, None, None
    if momentum is not None:
        mom_code = _row_code(momentum, "momentum")
        _need_shape(momentum, "momentum", momentum.dtype, dev, shape)
        mp = np_ = momentum.data_ptr()
        if new_momentum is not None:
            _need_shape(new_momentum, "new_momentum", momentum.dtype, dev, shape)
            np_ = new_momentum.data_ptr()
    flat = _coefficients(coeffs, steps)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    else:
        _need_shape(out, "out", torch.bfloat16, dev, shape)
    if ws is None:
        ws = workspace(orthogonalize_workspace_size(L, rows, cols), dev)
    _lib.check(_lib.load().eas_orthogonalize(
        grad.data_ptr(), code, mp, np_, mom_code, L, rows, cols, beta, 1 if nesterov else 0,
        flat.buffer_info()[0], steps, eps, scale, out.data_ptr(), *_ws_args(ws, dev), _stream(dev)))
    return out


def orthogonalize(grad, steps: int = 5, coeffs=NEWTON_SCHULZ, eps: float = 1e-7, scale: float = 1.0,
                  ws=None, out=None):
    """scale times the orthogonalised matrix (or stack of matrices, [L, rows, cols]):
    grad over its 2-norm, then `steps` Newton-Schulz products.  bf16.

    coeffs: (a, b, c) of every step, or one triple for each."""
    return _orthogonalize(grad, None, None, 0.0, False, steps, coeffs, eps, scale, ws, out)


def muon_update(grad, momentum, beta: float = 0.95, nesterov: bool = True, steps: int = 5,
                coeffs=NEWTON_SCHULZ, eps: float = 1e-7, scale: float = 1.0, new_momentum=None,
                ws=None, out=None):
    """One Muon update: momentum = beta momentum + (1 - beta) grad, in place or into
    new_momentum; returns scale times the orthogonalised momentum (with nesterov, of
    beta momentum + (1 - beta) grad) in bf16, for param.sub_(update, alpha=lr).

    grad and momentum are [rows, cols] or a stack [L, rows, cols], each bf16 or fp32."""
    if momentum is None:
        raise ValueError("momentum must be a tensor (orthogonalize takes none)")
    return _orthogonalize(grad, momentum, new_momentum, beta, nesterov, steps, coeffs, eps, scale,
                          ws, out)
