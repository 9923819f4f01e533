"""The two ends of a training step together: scores of logits that exist and their
gradient, clipping, the orthogonalised update; and the scores against the LM head's."""
import math
import os
import sys

import numpy as np
import pytest
import torch

import entropy_active_span_gb300 as eas
import oracle

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def rel(a, b):
    return float(np.linalg.norm(f64(a) - np.asarray(b)) / np.linalg.norm(b))


def test_scores_agree_with_the_lm_head():
    """The same definitions: on the logits that the LM head never writes down, its
    logprob, entropy and lse.  fp32 logits of a torch product and the LM head's own sums
    differ by the rounding of H products, 2^-24 sqrt(H) |z|; twice that of the largest z."""
    T, H, V = 300, 256, 3000
    g = torch.Generator().manual_seed(0)
    h = torch.randn(T, H, generator=g).bfloat16().cuda()
    w = (torch.randn(V, H, generator=g) * 0.3).bfloat16().cuda()
    t = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    mask = (torch.rand(T, generator=g) < 0.7).to(torch.uint8).cuda()
    spans, n = eas.build_active_spans(mask)
    lp, ent, lse = eas.lmhead_fwd(h, w, t, mask, spans, n)
    z = (h.double() @ w.double().t()).float()
    slp, sent, slse, top, ids = eas.token_logprobs_fwd(z, t, 5, mask=mask)
    tol = 2e-3
    for a, b in ((lp, slp), (ent, sent), (lse, slse)):
        assert float((a - b).abs().max()) <= tol
    on = mask.bool()
    assert torch.equal(ids[on, 0].long(), z[on].argmax(-1)) and (ids[~on] == -1).all()
    assert (top[on, 0] >= slp[on]).all()


# bf16 gradients of the loss (2^-8 each) summed over T tokens in a torch product, rounded
# to bf16 again, and what the orthogonalisation makes of an error of that size: about
# three times its share of the norm, beside its own 3.4e-3.
FRO = 0.03


def test_a_distillation_step():
    """loss = -sum logprob(target) - beta entropy - sum over the student's alternatives of
    weights logprob; dW = dlogits^T h; clipped; W -= lr muon(dW)."""
    T, H, V, k, beta, lr = 400, 128, 2000, 4, 0.05, 0.02
    g = torch.Generator().manual_seed(1)
    h = torch.randn(T, H, generator=g).cuda()
    w = (torch.randn(V, H, generator=g) * 0.2).cuda()
    t = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8).cuda()
    weights = torch.rand(T, k, generator=g).cuda() * mask[:, None]
    mom = (torch.randn(V, H, generator=g) * 1e-2).cuda()

    logits = (h @ w.t()).requires_grad_()
    lp, ent, top, ids = eas.fused_token_logprobs(logits, t, k, mask=mask)
    loss = -(lp.sum() + beta * ent.sum() + (weights * top).sum())
    loss.backward()
    dw = (logits.grad.t() @ h).contiguous()
    norm = eas.clip_grad_norm([dw], 1.0)
    before = mom.clone()
    step = eas.muon_update(dw, mom, scale=math.sqrt(V / H))
    new = w - lr * step.float()

    # the same in 64 bits
    z = f64(h) @ f64(w).T
    on = f64(mask) != 0
    rlp, rent, rlse, rtop, rids = oracle.token_scores(z, t.cpu().numpy()[:, None], k, mask=on)
    assert np.array_equal(ids.cpu().numpy(), rids)
    tokens = np.concatenate([t.cpu().numpy()[:, None], rids], 1)
    gl = -np.concatenate([np.ones((T, 1)), f64(weights)], 1)
    dz = oracle.token_scores_grad(gl, np.full(T, -beta), z, tokens, rlse, rent, mask=on)
    rloss = -(rlp.sum() + beta * rent.sum() + (f64(weights) * rtop).sum())
    assert abs(loss.item() - rloss) <= 1e-4 * abs(rloss)
    rnorm, (rdw,) = oracle.clip_grads([dz.T @ f64(h)], 1.0)
    assert abs(float(norm) - rnorm) <= 1e-4 * rnorm and rel(dw, rdw) <= 1e-4
    rmom, u = oracle.momentum_update(rdw, f64(before), 0.95, True)
    ref = math.sqrt(V / H) * oracle.orthogonalize(u, [eas.NEWTON_SCHULZ] * 5, 1e-7)
    assert rel(mom, rmom) <= 1e-4 and rel(step, ref) <= FRO
    assert rel(new, f64(w) - lr * ref) <= FRO


def test_calls_on_two_streams_at_once():
    """Kernels whose CTAs wait for one another beside each other and beside the LM head's."""
    g = torch.randn(2048, 1500, device="cuda").bfloat16()
    small = torch.randn(40, 100, 120, device="cuda")
    x = torch.randn(600, 40000, device="cuda").bfloat16()
    ref = eas.orthogonalize(g), eas.orthogonalize(small), eas.token_logprobs_fwd(x, None, 8)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = []
    for i in range(12):
        with torch.cuda.stream(streams[i % 4]):
            outs.append((eas.orthogonalize(g), eas.orthogonalize(small), eas.token_logprobs_fwd(x, None, 8)))
    torch.cuda.synchronize()
    for a, b, c in outs:
        assert torch.equal(a, ref[0]) and torch.equal(b, ref[1])
        assert all(torch.equal(p, q) for p, q in zip(c[1:], ref[2][1:]))


def test_a_step_captured_and_replayed():
    T, V, H = 64, 3000, 200
    logits = torch.randn(T, V, device="cuda").bfloat16()
    t = torch.randint(0, V, (T,), dtype=torch.int32, device="cuda")
    h = torch.randn(T, H, device="cuda").bfloat16()
    mom = torch.zeros(V, H, device="cuda")

    def step():
        lp, ent, lse, top, ids = eas.token_logprobs_fwd(logits, t, 6)
        d = eas.token_logprobs_bwd(torch.full_like(lp, -1.0), None, logits, t, lse, ent)
        dw = (d.t() @ h).contiguous()
        eas.clip_grad_norm([dw], 1.0)
        return lp, ids, eas.muon_update(dw, mom)

    eager = step()
    after = mom.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(2):
        mom.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(mom, after) and all(torch.equal(a, b) for a, b in zip(held, eager))


def test_the_example_steps_with_muon():
    import tied_step as ex
    m, b = ex.make_model(600, 256), ex.make_batch(512, 600)
    buf = torch.zeros_like(m.layer, dtype=torch.float32)
    before = m.layer.clone()
    loss, norm = ex.step(m, b, momentum=buf)
    assert torch.isfinite(loss) and torch.isfinite(norm) and float(buf.abs().max()) > 0
    assert not torch.equal(before, m.layer) and torch.isfinite(m.layer).all()
    lp, ids = ex.alternatives(m, b, 4)
    assert ids.shape == (512, 4) and (ids[~b["mask"].bool()] == -1).all() and (lp <= 0).all()
