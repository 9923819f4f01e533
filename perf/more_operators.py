"""Cases of the operators at the two ends of a training step: the scores of logits
that exist (log probabilities of given tokens, entropy, top alternatives) with
their gradient, and the orthogonalised update of a matrix behind the clipping.

Each case runs either in plain torch operations (own = False) or through the
package's entry points (own = True) on the same inputs."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
COEFFS = (3.4445, -4.7750, 2.0315)
STEPS, BETA, EPS = 5, 0.95, 1e-7


def listed():
    return [
        # the sampled token of one generation step with its 8 alternatives: latency
        {"name": "score_token", "op": "score", "N": 1, "V": 128256, "M": 1, "k": 8, "dtype": "bf16",
         "scale": 1.0, "mask": "none", "constrained": False},
        # a decoding batch in fp32 at a temperature, a quarter of it under a grammar
        {"name": "score_decode_64", "op": "score", "N": 64, "V": 152064, "M": 1, "k": 20,
         "dtype": "fp32", "scale": 1.25, "mask": "none", "constrained": True},
        # several given tokens a row and many alternatives, rows of odd width
        {"name": "score_odd_fp32", "op": "score", "N": 777, "V": 32003, "M": 5, "k": 64,
         "dtype": "fp32", "scale": 1.0, "mask": "none", "constrained": False},
        # the responses of 16 sequences of 1024 tokens behind their loss mask
        {"name": "score_rl_16k", "op": "score", "N": 16384, "V": 128256, "M": 1, "k": 8,
         "dtype": "bf16", "scale": 1.0, "mask": "rl_1024", "constrained": False},
        # the smallest configuration's rows: latency
        {"name": "score_bwd_small_fp32", "op": "score_bwd", "N": 256, "V": 1024, "M": 1,
         "dtype": "fp32", "scale": 1.0, "mask": "none", "constrained": False},
        # distillation on a teacher's 20 alternatives
        {"name": "score_bwd_distill_2k", "op": "score_bwd", "N": 2048, "V": 152064, "M": 20,
         "dtype": "fp32", "scale": 1.0, "mask": "none", "constrained": False},
        # the policy gradient and the entropy bonus behind a loss mask
        {"name": "score_bwd_rl_16k", "op": "score_bwd", "N": 16384, "V": 128256, "M": 1,
         "dtype": "bf16", "scale": 1.0, "mask": "rl_1024", "constrained": False},
        # the twelve matrices of a small fp32 model, stacked: latency
        {"name": "muon_small_fp32", "op": "muon", "L": 12, "n": 128, "m": 128, "dtype": "fp32",
         "momentum": "fp32"},
        # one matrix of odd sizes, without a momentum
        {"name": "muon_odd_fp32", "op": "muon", "L": 1, "n": 1003, "m": 777, "dtype": "fp32",
         "momentum": "none"},
        # a stack of eight smaller matrices
        {"name": "muon_stack_8", "op": "muon", "L": 8, "n": 1024, "m": 2048, "dtype": "bf16",
         "momentum": "bf16"},
        # a square matrix of a layer: bf16 gradient, fp32 momentum
        {"name": "muon_4k", "op": "muon", "L": 1, "n": 4096, "m": 4096, "dtype": "bf16",
         "momentum": "fp32"},
        # a layer's widening matrix, taller than wide
        {"name": "muon_tall_16k", "op": "muon", "L": 1, "n": 16384, "m": 4096, "dtype": "bf16",
         "momentum": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "score_bwd", "muon"])
    if op == "muon":
        n = rng.choice([128, 320, 1003, 1088, 4096, 5120, _log(rng, 32, 5120), _log(rng, 32, 5120)])
        m = rng.choice([128, 320, 777, 4096, _log(rng, 32, 8192), _log(rng, 32, 8192)])
        most = min(12, max(1, int(4e11 / _muon_flops(n, m))))
        return {"op": op, "L": rng.randint(1, most), "n": n, "m": m,
                "dtype": rng.choice(["bf16", "bf16", "fp32"]),
                "momentum": rng.choice(["none", "fp32", "fp32", "bf16"])}
    V = rng.choice([1000, 32003, 32768, 128256, 129280, 152064, _log(rng, 100, 160000)])
    N = _log(rng, 1, min(16384, (1 << 30) // V))
    masks = ["none", "none"] + ["rl_1024"] * 2 * (N >= 1024)
    c = {"op": op, "N": N, "V": V, "M": rng.choice([1, 1, 1, 2, 5, 20]),
         "dtype": rng.choice(["bf16", "bf16", "fp32"]), "scale": rng.choice([1.0, 1.0, 0.5, 1.25]),
         "mask": rng.choice(masks), "constrained": rng.random() < 0.3}
    if op == "score":
        c["k"] = rng.choice([0, 1, 5, 8, 20, 20, 64])
    return c


# ------------------------------------------------------------------ inputs

def _logits(case, g):
    """Logits of a model: a spread of values, half of the rows with a few tokens far
    above it; constrained: a quarter of the rows allow few tokens (-inf elsewhere).
    Also a likely token of each row."""
    N, V, dt = case["N"], case["V"], DTYPES[case["dtype"]]
    x = torch.randn((N, V), device="cuda", dtype=dt, generator=g).mul_(2.5)
    likely = torch.randint(0, V, (N, 4), device="cuda", generator=g)
    lift = 4.0 + 10.0 * torch.rand((N, 4), device="cuda", generator=g)
    lift[::2] *= 0.5
    x.scatter_(1, likely, lift.to(dt))
    if case["constrained"]:
        rows = x[::4]
        share = torch.rand((rows.shape[0], 1), device="cuda", generator=g).mul_(0.05)
        off = torch.rand(rows.shape, device="cuda", generator=g) >= share
        off.scatter_(1, likely[::4], False)
        rows.masked_fill_(off, -math.inf)
    return x, likely


def _mask(kind, n, g):
    """Prompt / response sequences; the responses are active."""
    if kind == "none":
        return None
    seq = int(kind[3:])
    pos = torch.arange(n, device="cuda")
    prompt = torch.randint(seq // 4, seq // 2 + 1, ((n + seq - 1) // seq,), device="cuda", generator=g)
    return (pos % seq >= prompt[pos // seq]).to(torch.uint8)


def _stats(x, scale):
    """lse and entropy as a forward left them, rounded to fp32."""
    lse = torch.empty(x.shape[0], device="cuda", dtype=torch.float32)
    ent = torch.empty_like(lse)
    step = max(1, (1 << 27) // x.shape[1])
    for a in range(0, x.shape[0], step):
        z = x[a:a + step].float() * scale
        top = z.amax(-1, keepdim=True)
        e = (z - top).exp()
        s = e.sum(-1, dtype=torch.float64)
        u = torch.where(e > 0, e * (z - top), 0.0).sum(-1, dtype=torch.float64)
        lse[a:a + step] = top[:, 0].double() + s.log()
        ent[a:a + step] = s.log() - u / s
    return lse, ent


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("score", "score_bwd"):
        N, V, M = case["N"], case["V"], case["M"]
        x, likely = _logits(case, g)
        tokens = torch.randint(0, V, (N, M), device="cuda", generator=g)
        pick = likely[:, torch.arange(M, device="cuda") % 4]
        often = torch.rand((N, M), device="cuda", generator=g) < 0.7
        often[::4] |= case["constrained"]
        tokens = torch.where(often, pick, tokens)
        if M > 1:                                      # fewer given tokens in some rows
            tokens[:, 1:][torch.rand((N, M - 1), device="cuda", generator=g) < 0.1] = -1
        st = {"case": case, "x": x, "tokens": tokens.to(torch.int32), "mask": _mask(case["mask"], N, g)}
        if case["op"] == "score_bwd":
            st["g_lp"] = torch.randn((N, M), device="cuda", generator=g)
            st["g_ent"] = torch.randn(N, device="cuda", generator=g).mul_(0.01)
            st["lse"], st["ent"] = _stats(x, case["scale"])
        return st
    L, n, m = case["L"], case["n"], case["m"]
    rank = min(32, n, m)
    left = torch.randn((L, n, rank), device="cuda", generator=g)
    left *= torch.logspace(0, -1.5, rank, device="cuda")
    right = torch.randn((L, rank, m), device="cuda", generator=g)
    grad = torch.randn((L, n, m), device="cuda", generator=g).mul_(0.1)
    grad.baddbmm_(left, right).mul_(1e-3)              # a few strong directions and noise
    st = {"case": case, "grad": grad.to(dt), "mom": None}
    if case["momentum"] != "none":
        mom = torch.randn((L, n, m), device="cuda", generator=g).mul_(2e-4)
        st["mom"] = mom.baddbmm_(left, right, alpha=1e-3).to(DTYPES[case["momentum"]])
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        return _run_own(case["op"], case, st)
    if case["op"] == "score":
        return _score(case, st)
    if case["op"] == "score_bwd":
        return _score_bwd(case, st)
    return _muon(case, st)


def _run_own(op, case, st):
    import entropy_active_span_gb300 as eas
    if op == "score":
        lp, ent, lse, top, ids = eas.token_logprobs_fwd(st["x"], st["tokens"], top_k=case["k"],
                                                        scale=case["scale"], mask=st["mask"])
        out = {"logprob": lp, "entropy": ent, "lse": lse}
        if case["k"]:
            out["top"], out["ids"] = top, ids
        return out
    if op == "score_bwd":
        return {"dx": eas.token_logprobs_bwd(st["g_lp"], st["g_ent"], st["x"], st["tokens"],
                                             st["lse"], st["ent"], scale=case["scale"],
                                             mask=st["mask"])}
    if st["mom"] is None:
        return {"update": eas.orthogonalize(st["grad"], steps=STEPS, coeffs=COEFFS, eps=EPS)}
    new = torch.empty_like(st["mom"])                  # the state stays for the next pass
    out = eas.muon_update(st["grad"], st["mom"], beta=BETA, nesterov=True, steps=STEPS,
                          coeffs=COEFFS, eps=EPS, new_momentum=new)
    return {"update": out, "momentum": new}


def _score(case, st):
    x, V, k = st["x"].float(), case["V"], case["k"]
    on = None if st["mask"] is None else st["mask"].bool()[:, None]
    z = x * case["scale"]
    top = z.amax(-1, keepdim=True)
    e = (z - top).exp()
    s = e.sum(-1, keepdim=True)
    u = torch.where(e > 0, e * (z - top), 0.0).sum(-1, keepdim=True)
    logs = s.log()
    real = st["tokens"] >= 0
    lp = z.gather(1, st["tokens"].clamp(min=0).long()) - top - logs
    lp = torch.where(real, lp, 0.0)
    lse, ent = top + logs, logs - u / s
    out = {"logprob": lp, "entropy": ent, "lse": lse}
    if k:
        # order of the values, then of the columns, as one whole number
        bits = (x + 0.0).view(torch.int32)             # -0 counts as 0
        rank = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        key = rank * (1 << 32) + (0xFFFFFFFF - torch.arange(V, device="cuda"))
        ids = 0xFFFFFFFF - (key.topk(k, dim=-1).values & 0xFFFFFFFF)
        out["top"], out["ids"] = z.gather(1, ids) - top - logs, ids.to(torch.int32)
    if on is not None:
        out = {n: torch.where(on, v, -1 if n == "ids" else 0) for n, v in out.items()}
    return {n: v[:, 0] if n in ("entropy", "lse") else v for n, v in out.items()}


def _score_bwd(case, st):
    scale, tokens = case["scale"], st["tokens"]
    g = torch.where(tokens >= 0, st["g_lp"], 0.0)
    logp = st["x"].float() * scale - st["lse"][:, None]
    p = logp.exp()
    w = g.sum(-1, keepdim=True) + st["g_ent"][:, None] * (logp + st["ent"][:, None])
    d = torch.where(p > 0, -p * w, 0.0)
    d.scatter_add_(1, tokens.clamp(min=0).long(), g)
    d *= scale
    if st["mask"] is not None:
        d = torch.where(st["mask"].bool()[:, None], d, 0.0)
    return {"dx": d.to(st["x"].dtype)}


def _muon(case, st):
    g = st["grad"].float()
    out = {}
    if st["mom"] is not None:
        mom = BETA * st["mom"].float() + (1 - BETA) * g
        out["momentum"] = mom.to(st["mom"].dtype)
        g = (1 - BETA) * g + BETA * mom
    x = g / (g.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
    tall = case["n"] > case["m"]
    if tall:
        x = x.mT.contiguous()
    a, b, c = COEFFS
    for _ in range(STEPS):
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    out["update"] = (x.mT if tall else x).to(torch.bfloat16).contiguous()
    return out


# ------------------------------------------------------------------ floors

def _size(name):
    return 2 if name == "bf16" else 4


def _active(case):
    return 1.0 if case["mask"] == "none" else 0.625


def _muon_flops(n, m):
    """The two symmetric products of a step count once."""
    n, m = min(n, m), max(n, m)
    return STEPS * (3 * n * n * m + n ** 3)


def work(case):
    if case["op"] == "muon":
        nm = case["L"] * case["n"] * case["m"]
        mom = 0 if case["momentum"] == "none" else 2 * _size(case["momentum"])
        return {"bytes": nm * (_size(case["dtype"]) + 2 + mom),
                "flops": case["L"] * _muon_flops(case["n"], case["m"])}
    N, V, M, a = case["N"], case["V"], case["M"], _active(case)
    n, e, m = N * V, _size(case["dtype"]), N * (case["mask"] != "none")
    if case["op"] == "score":
        return {"bytes": a * n * e + m + N * (8 * M + 8 + 8 * case["k"]), "flops": 7 * a * n}
    return {"bytes": (1 + a) * n * e + m + a * N * (8 * M + 12), "flops": 8 * a * n}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions in 64 bits, a block of rows or a matrix at a time."""
    st = prepare(case, seed)
    f64 = dict(device="cuda", dtype=torch.float64)
    if case["op"] == "muon":
        L, n, m = case["L"], case["n"], case["m"]
        a, b, c = COEFFS
        out = {"update": torch.empty((L, n, m), **f64)}
        if st["mom"] is not None:
            out["momentum"] = torch.empty((L, n, m), **f64)
        for i in range(L):
            u = st["grad"][i].double()
            if st["mom"] is not None:
                out["momentum"][i] = st["mom"][i].double() * BETA + u * (1 - BETA)
                u = u * (1 - BETA) + out["momentum"][i] * BETA
            u /= torch.linalg.matrix_norm(u) + EPS
            for _ in range(STEPS):
                # the products from the shorter side
                if n <= m:
                    q = u @ u.T
                    u = a * u + (b * q + c * q @ q) @ u
                else:
                    q = u.T @ u
                    u = a * u + u @ (b * q + c * q @ q)
            out["update"][i] = u
        return out
    N, V, M, scale = case["N"], case["V"], case["M"], case["scale"]
    on = torch.ones(N, device="cuda", dtype=torch.bool) if st["mask"] is None else st["mask"].bool()
    step = max(1, (1 << 26) // V)
    if case["op"] == "score_bwd":
        dx = torch.zeros((N, V), **f64)
        for a in range(0, N, step):
            r = slice(a, a + step)
            logp = st["x"][r].double() * scale - st["lse"][r, None].double()
            p, t = logp.exp(), st["tokens"][r].long()
            logp.masked_fill_(p == 0, 0.0)
            g = st["g_lp"][r].double() * (t >= 0)
            d = dx[r]
            d.sub_(p * g.sum(1, keepdim=True))
            d.sub_(p * (logp + st["ent"][r, None].double()) * st["g_ent"][r, None].double())
            d.scatter_add_(1, t.clamp(min=0), g)
            d.mul_(scale).mul_(on[r, None])
        return {"dx": dx}
    k = case["k"]
    out = {"logprob": torch.zeros((N, M), **f64), "entropy": torch.zeros(N, **f64),
           "lse": torch.zeros(N, **f64)}
    if k:
        out["top"], out["ids"] = torch.zeros((N, k), **f64), None
    for a in range(0, N, step):
        r = slice(a, a + step)
        z, t, keep = st["x"][r].double() * scale, st["tokens"][r].long(), on[r]
        lse = torch.logsumexp(z, 1)
        logp = z - lse[:, None]
        out["lse"][r] = lse * keep
        out["entropy"][r] = -(logp.exp() * logp.clamp(min=-1e300)).sum(1) * keep
        lp = logp.gather(1, t.clamp(min=0))
        out["logprob"][r] = torch.where((t >= 0) & keep[:, None], lp, 0.0)
        if k:
            out["top"][r] = torch.where(keep[:, None], logp.sort(1, descending=True).values[:, :k], 0.0)
    return out
