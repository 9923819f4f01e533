"""One RL training step of a small language model with tied embeddings, every
operator around its one dense layer from this package:

    x  = scale E[ids]                      embed_fwd
    h  = tanh(x W)                         (torch)
    y  = rmsnorm(x + h) g                  rmsnorm_fwd, loss mask, optional e4m3 codes
    logprob, entropy = lm_head(y, E)       lmhead_fwd or lmhead_fwd_fp8
    loss = -sum over active tokens of advantage logprob + beta entropy

and back: lmhead_bwd -> rmsnorm_bwd -> the layer -> embed_bwd, which adds its
sums to the LM head's gradient of E, then clip_grad_norm over all gradients and
a plain SGD update, or with --muon the orthogonalised one of the dense layer.  At the
end the model's own alternatives at the first active tokens, from logits that exist
(token_logprobs_fwd).  Run it on a GPU:

    python examples/tied_step.py [--fp8] [--muon] [--steps N]
"""
from __future__ import annotations

import argparse
import dataclasses
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import entropy_active_span_gb300 as eas  # noqa: E402

EPS = 1e-6


@dataclasses.dataclass
class Model:
    table: torch.Tensor     # [V, H] bf16, embedding and LM head
    layer: torch.Tensor     # [H, H] bf16
    gain: torch.Tensor      # [H] bf16

    @property
    def scale(self) -> float:
        return math.sqrt(self.table.shape[1])


def make_model(V: int, H: int, seed: int = 0) -> Model:
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(shape, generator=g) * std).bfloat16().cuda()

    return Model(normal(V, H, std=0.1), normal(H, H, std=H ** -0.5),
                 (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda())


def make_batch(T: int, V: int, seed: int = 0) -> dict:
    """Token ids (the last 5 % are padding, id -1), the next tokens as targets, a
    loss mask that leaves the prompt out, and advantages."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    targets = ids.roll(-1).contiguous()
    real = T - T // 20
    mask = torch.zeros(T, dtype=torch.uint8)
    mask[T // 4:real - 1] = 1
    ids[real:] = -1
    return {"ids": ids.cuda(), "targets": targets.clamp(min=0).cuda(), "mask": mask.cuda(),
            "advantage": torch.randn(T, generator=g).cuda()}


def gradients(m: Model, batch: dict, beta: float = 0.01, fp8: bool = False):
    """(loss, {name: fp32 or bf16 gradient}) of one batch, by the package's calls."""
    ids, targets, mask, adv = (batch[k] for k in ("ids", "targets", "mask", "advantage"))
    V = m.table.shape[0]
    spans, num_spans = eas.build_active_spans(mask)
    x = eas.embed_fwd(ids, m.table, m.scale)
    h = torch.tanh(x @ m.layer)
    y, q, q_scale, s = eas.rmsnorm_fwd(h, m.gain, EPS, residual=x, mask=mask, want_e4m3=fp8)
    if fp8:
        t8, t_scale = eas.quantize_rows_e4m3(m.table)
        lp, ent, lse = eas.lmhead_fwd_fp8(q, q_scale, t8, t_scale, targets, mask, spans, num_spans)
    else:
        lp, ent, lse = eas.lmhead_fwd(y, m.table, targets, mask, spans, num_spans)
    loss = -(adv * lp + beta * ent).sum()
    g_lp, g_ent = -adv, torch.full_like(adv, -beta)
    if fp8:
        dy, dtable = eas.lmhead_bwd_fp8(g_lp, g_ent, y, m.table, q, q_scale, t8, t_scale, targets,
                                        mask, spans, num_spans, lse, ent)
    else:
        dy, dtable = eas.lmhead_bwd(g_lp, g_ent, y, m.table, targets, mask, spans, num_spans, lse, ent)
    ds, dgain = eas.rmsnorm_bwd(dy, s, m.gain, EPS, mask=mask)
    dpre = ds * (1 - h * h)
    dx = torch.addmm(ds, dpre, m.layer.t())
    dlayer = x.t() @ dpre
    eas.embed_bwd(ids, dx, V, m.scale, accumulate=True, dweight=dtable)
    return loss, {"table": dtable, "layer": dlayer.contiguous(), "gain": dgain}


def step(m: Model, batch: dict, lr: float = 0.05, max_norm: float = 1.0, fp8: bool = False,
         momentum: torch.Tensor | None = None):
    """One update; returns (loss, gradient norm before clipping) on the device.
    momentum: [H, H] fp32, kept by the caller; with it the dense layer's update is
    Muon's, of the size that a layer of its shape takes."""
    loss, grads = gradients(m, batch, fp8=fp8)
    clipped = {k: torch.empty_like(getattr(m, k)) for k in grads}     # in the weights' type
    norm = eas.clip_grad_norm(list(grads.values()), max_norm, out=list(clipped.values()))
    if momentum is not None:
        clipped["layer"] = eas.muon_update(clipped["layer"], momentum,
                                           scale=0.2 * math.sqrt(max(m.layer.shape)))
    for k, g in clipped.items():
        getattr(m, k).sub_(g, alpha=lr)
    return loss, norm


def alternatives(m: Model, batch: dict, k: int):
    """(log probabilities [T, k], token ids [T, k]) of the k likeliest next tokens at the
    active positions, as a sampler reports them: from the logits themselves."""
    x = eas.embed_fwd(batch["ids"], m.table, m.scale)
    y, _, _, _ = eas.rmsnorm_fwd(torch.tanh(x @ m.layer), m.gain, EPS, residual=x, mask=batch["mask"],
                                 want_sum=False)
    _, _, _, top, ids = eas.token_logprobs_fwd(y @ m.table.t(), None, k, mask=batch["mask"])
    return top, ids


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--fp8", action="store_true", help="e4m3 logits")
    ap.add_argument("--muon", action="store_true", help="orthogonalised update of the dense layer")
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    m, batch = make_model(4096, 512), make_batch(2048, 4096)
    momentum = torch.zeros(m.layer.shape, device="cuda") if a.muon else None
    for i in range(a.steps):
        loss, norm = step(m, batch, fp8=a.fp8, momentum=momentum)
        print(f"step {i}: loss {float(loss):.3f}  gradient norm {float(norm):.3f}")
    top, ids = alternatives(m, batch, 3)
    for t in batch["mask"].nonzero()[:3, 0].tolist():
        print(f"token {t}: " + "  ".join(f"{i} ({p:.2f})" for i, p in zip(ids[t].tolist(), top[t].tolist())))


if __name__ == "__main__":
    main()
