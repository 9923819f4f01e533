"""Cases of the operators around the LM head: the residual RMS norm with an
e4m3 output and its backward, the scaled embedding lookup and its gradient,
and the global gradient norm with clipping.

Each case runs either in plain torch operations (own = False) or through the
package's entry points (own = True) on the same inputs."""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # a single token of a generation step through the final norm: latency
        {"name": "norm_token", "op": "norm", "R": 1, "H": 4096, "dtype": "bf16", "residual": True,
         "e4m3": True, "mask": "none"},
        # the final norm of an RL batch of 16 x 1024 tokens, feeding the e4m3 LM head
        {"name": "norm_rl_16k", "op": "norm", "R": 16384, "H": 4096, "dtype": "bf16",
         "residual": True, "e4m3": True, "mask": "rl_1024"},
        # the same on 32 sequences of 8192 tokens: the largest one-GPU batch
        {"name": "norm_long_256k", "op": "norm", "R": 262144, "H": 8192, "dtype": "bf16",
         "residual": True, "e4m3": True, "mask": "rl_8192"},
        # an odd width in fp32 (no row but the first is aligned), every row active
        {"name": "norm_bwd_odd_fp32", "op": "norm_bwd", "R": 777, "H": 1003, "dtype": "fp32",
         "residual": False, "mask": "none"},
        # the backward of a norm inside the model: the residual stream's gradient is added
        {"name": "norm_bwd_packed_64k", "op": "norm_bwd", "R": 65536, "H": 5120, "dtype": "bf16",
         "residual": True, "mask": "none"},
        # the backward of the final norm behind a loss mask with 10 % active tokens
        {"name": "norm_bwd_sparse_128k", "op": "norm_bwd", "R": 131072, "H": 7168, "dtype": "bf16",
         "residual": False, "mask": "sparse"},
        # the tokens of one decoding step of 16 sequences: latency
        {"name": "embed_tokens_16", "op": "embed", "T": 16, "H": 4096, "V": 128256,
         "dtype": "bf16", "ids": "uniform", "pad": 0.0},
        # packed bins with their alignment padding
        {"name": "embed_packed_64k", "op": "embed", "T": 65536, "H": 5120, "V": 152064,
         "dtype": "bf16", "ids": "zipf", "pad": 0.1},
        # far fewer tokens than vocabulary rows: most of the gradient is zeros
        {"name": "embed_bwd_rl_16k", "op": "embed_bwd", "T": 16384, "H": 4096, "V": 128256,
         "dtype": "bf16", "ids": "uniform", "pad": 0.0},
        # Zipf-distributed tokens: a few rows collect thousands of tokens
        {"name": "embed_bwd_sparse_128k", "op": "embed_bwd", "T": 131072, "H": 7168, "V": 129280,
         "dtype": "bf16", "ids": "zipf", "pad": 0.1},
        # the gradients of a small fp32 model (1024 x 128 vocabulary): latency
        {"name": "clip_small_fp32", "op": "clip", "V": 1024, "H": 128, "mats": 12, "odd": 5,
         "dtype": "fp32", "out": "fp32", "max_norm": 1.0},
        # the fp32 dW of the LM head and the bf16 gradients of the layers below it,
        # clipped into the bf16 gradients that the optimiser reads
        {"name": "clip_rl_16k", "op": "clip", "V": 128256, "H": 4096, "mats": 48, "odd": 5,
         "dtype": "bf16", "out": "bf16", "max_norm": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "embed", "embed_bwd", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    H = rng.choice([128, 320, 1003, 1088, 4096, 5120, 7168, 8192, _log(rng, 64, 8192)])
    if op in ("norm", "norm_bwd"):
        # at most 65536 x 8192 elements, a quarter of the largest listed case
        R = _log(rng, 1, min(131072, (1 << 29) // H))
        masks = ["none"] + ["rl_1024", "sparse"] * (R >= 1024) + ["rl_8192"] * (R >= 8192)
        c = {"op": op, "R": R, "H": H, "dtype": dtype, "residual": rng.random() < 0.7,
             "mask": rng.choice(masks)}
        if op == "norm":
            c["e4m3"] = rng.random() < 0.7
        return c
    if op in ("embed", "embed_bwd"):
        T, V = _log(rng, 1, min(131072, (1 << 29) // H)), _log(rng, 1000, 152064)
        return {"op": op, "T": T, "H": H, "V": V, "dtype": dtype,
                "ids": rng.choice(["uniform", "zipf"]),
                "pad": rng.choice([0.0, 0.1]) if T >= 128 else 0.0}
    return {"op": "clip", "V": _log(rng, 100, 40000), "H": rng.choice([128, 320, 1003, 1088, 4096]),
            "mats": rng.randrange(1, 49), "odd": rng.randrange(0, 8), "dtype": dtype,
            "out": rng.choice(["bf16", "fp32"]), "max_norm": rng.choice([0.5, 1.0, 1e4])}


# ------------------------------------------------------------------ inputs

def _mask(kind, n, g):
    """Loss masks: prompt / response sequences, or short active runs far apart."""
    if kind == "none":
        return None
    pos = torch.arange(n, device="cuda")
    if kind == "sparse":
        runs = n // 16 + 2
        gaps = torch.randint(1, 648, (runs,), device="cuda", generator=g)
        acts = torch.randint(8, 65, (runs,), device="cuda", generator=g)
        ends = torch.stack([gaps, acts], 1).reshape(-1).cumsum(0)
        return (torch.searchsorted(ends, pos, right=True) % 2).to(torch.uint8)
    seq = int(kind[3:])
    lo, hi = (256, 512) if seq == 1024 else (2458, 4096)
    prompt = torch.randint(lo, hi + 1, ((n + seq - 1) // seq,), device="cuda", generator=g)
    return (pos % seq >= prompt[pos // seq]).to(torch.uint8)


def _normal(shape, dtype, std, g):
    return torch.randn(shape, device="cuda", dtype=dtype, generator=g).mul_(std)


def _ids(case, g):
    T, V = case["T"], case["V"]
    if case["ids"] == "zipf":
        cdf = (torch.arange(1, V + 1, device="cuda", dtype=torch.float64) ** -1.1).cumsum(0)
        u = torch.rand(T, device="cuda", dtype=torch.float64, generator=g) * cdf[-1]
        ids = torch.searchsorted(cdf, u, right=True).clamp_(max=V - 1)
    else:
        ids = torch.randint(0, V, (T,), device="cuda", generator=g)
    ids[torch.rand(T, device="cuda", generator=g) < case["pad"]] = -1   # alignment padding
    return ids.to(torch.int32)


def _clip_shapes(case):
    """The LM head's gradient in fp32, then matrices and vectors of odd length."""
    V, H = case["V"], case["H"]
    return [(V, H)] + [(H, H)] * case["mats"] + [(H + 1 + 2 * i,) for i in range(case["odd"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, H, dt = case["op"], case["H"], DTYPES[case["dtype"]]
    if op in ("norm", "norm_bwd"):
        R = case["R"]
        st = {"case": case, "w": _normal((H,), torch.float32, 0.1, g).add_(1.0).to(dt),
              "mask": _mask(case["mask"], R, g)}
        if op == "norm":
            st["x"] = _normal((R, H), dt, 1.0, g)
            st["r"] = _normal((R, H), dt, 2.0, g) if case["residual"] else None
        else:
            st["s"] = _normal((R, H), dt, 2.0, g)
            st["dy"] = _normal((R, H), dt, 1e-2, g)
            st["ds"] = _normal((R, H), dt, 1e-2, g) if case["residual"] else None
        return st
    if op in ("embed", "embed_bwd"):
        st = {"case": case, "ids": _ids(case, g), "scale": math.sqrt(H)}
        if op == "embed":
            st["table"] = _normal((case["V"], H), dt, 0.02, g)
        else:
            st["dout"] = _normal((case["T"], H), dt, 1e-2, g)
        return st
    # the first gradient is the LM head's, accumulated in fp32
    shapes = _clip_shapes(case)
    grads = [_normal(s, dt if i else torch.float32, 1e-3 * (1 + i % 3), g)
             for i, s in enumerate(shapes)]
    outs = [torch.empty(s, device="cuda", dtype=DTYPES[case["out"]]) for s in shapes]
    return {"case": case, "grads": grads, "outs": outs}


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        return _run_own(case["op"], case, st)
    return _run_plain(case["op"], case, st)


def _run_own(op, case, st):
    import entropy_active_span_gb300 as eas
    if op == "norm":
        y, q, scale, s = eas.rmsnorm_fwd(st["x"], st["w"], EPS, residual=st["r"], mask=st["mask"],
                                         want_e4m3=case["e4m3"])
        out = {"y": y}
        if case["residual"]:
            out["s"] = s
        if case["e4m3"]:
            out["q"], out["scale"] = q.view(torch.float8_e4m3fn), scale
        return out
    if op == "norm_bwd":
        dx, dw = eas.rmsnorm_bwd(st["dy"], st["s"], st["w"], EPS, ds=st["ds"], mask=st["mask"])
        return {"dx": dx, "dw": dw}
    if op == "embed":
        return {"out": eas.embed_fwd(st["ids"], st["table"], st["scale"])}
    if op == "embed_bwd":
        return {"dw": eas.embed_bwd(st["ids"], st["dout"], case["V"], st["scale"])}
    norm = eas.clip_grad_norm(st["grads"], case["max_norm"], out=st["outs"])
    return {"norm": norm, "grads": st["outs"]}


def _run_plain(op, case, st):
    if op == "norm":
        x, dt = st["x"], st["x"].dtype
        s = x.float() if st["r"] is None else x.float() + st["r"].float()
        y = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS) * st["w"].float()
        if st["mask"] is not None:
            y = torch.where(st["mask"].bool()[:, None], y, 0.0)
        out = {"y": y.to(dt)}
        if case["residual"]:
            out["s"] = s.to(dt)
        if case["e4m3"]:
            amax = y.abs().amax(-1)
            some = amax > 0
            inv = torch.where(some, 448.0 / amax, 1.0)
            out["scale"] = torch.where(some, amax / 448.0, 1.0)
            out["q"] = (y * inv[:, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        return out
    if op == "norm_bwd":
        dt, H = st["s"].dtype, case["H"]
        s, dy, w = st["s"].float(), st["dy"].float(), st["w"].float()
        if st["mask"] is not None:
            dy = torch.where(st["mask"].bool()[:, None], dy, 0.0)
        rstd = torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS)
        g = dy * w
        dx = rstd * (g - s * ((g * s).sum(-1, keepdim=True) * rstd * rstd / H))
        if st["ds"] is not None:
            dx = dx + st["ds"].float()
        return {"dx": dx.to(dt), "dw": (dy * (s * rstd)).sum(0)}
    if op == "embed":
        ids = st["ids"]
        rows = st["table"][ids.clamp(min=0).long()].float() * st["scale"]
        return {"out": torch.where((ids >= 0)[:, None], rows, 0.0).to(st["table"].dtype)}
    if op == "embed_bwd":
        ids, V = st["ids"].long(), case["V"]
        # padding goes to a row of its own past the end
        dw = torch.zeros((V + 1, case["H"]), device="cuda", dtype=torch.float32)
        dw.index_add_(0, torch.where(ids >= 0, ids, V), st["dout"].float() * st["scale"])
        return {"dw": dw[:V]}
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]]).sum().sqrt()
    coef = (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return {"norm": norm.float().reshape(1),
            "grads": [o.copy_(g.float() * coef) for g, o in zip(st["grads"], st["outs"])]}


# ------------------------------------------------------------------ floors

def _size(name):
    return 2 if name == "bf16" else 4


def _active(case):
    return {"none": 1.0, "rl_1024": 0.625, "rl_8192": 0.6, "sparse": 0.1}[case["mask"]]


def _distinct(case):
    """Expected number of vocabulary rows that the tokens touch."""
    T, V = case["T"] * (1.0 - case["pad"]), case["V"]
    if case["ids"] == "uniform":
        return V * -math.expm1(T * math.log1p(-1.0 / V)) if V > 1 else 1.0
    p = torch.arange(1, V + 1, dtype=torch.float64) ** -1.1
    return float(-torch.expm1(T * torch.log1p(-p / p.sum())).sum())


def work(case):
    op, H, e = case["op"], case["H"], _size(case["dtype"])
    if op == "norm":
        n = case["R"] * H
        b = n * e * (2 + 2 * case["residual"]) + H * e
        b += case["e4m3"] * (n + 4 * case["R"]) + (case["mask"] != "none") * case["R"]
        return {"bytes": b, "flops": n * (5 + 3 * case["e4m3"])}
    if op == "norm_bwd":
        n, a = case["R"] * H, _active(case)
        b = n * e * (2 * a + 1 + case["residual"]) + H * (e + 4)
        return {"bytes": b + (case["mask"] != "none") * case["R"], "flops": 13 * a * n}
    if op == "embed":
        n = case["T"] * H
        return {"bytes": 4 * case["T"] + e * (_distinct(case) * H + n), "flops": n}
    if op == "embed_bwd":
        n = case["T"] * H * (1.0 - case["pad"])
        return {"bytes": 4 * case["T"] + e * n + 4 * case["V"] * H, "flops": n}
    sizes = [math.prod(s) for s in _clip_shapes(case)]
    return {"bytes": 4 * sizes[0] + e * sum(sizes[1:]) + _size(case["out"]) * sum(sizes) + 4,
            "flops": 3 * sum(sizes)}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions in 64 bits, a block of rows or a tensor at a time."""
    st = prepare(case, seed)
    op, H = case["op"], case["H"]
    f64 = dict(device="cuda", dtype=torch.float64)
    if op in ("norm", "norm_bwd"):
        R = case["R"]
        on = torch.ones(R, 1, **f64) if st["mask"] is None else st["mask"].double()[:, None]
        w = st["w"].double()
        step = max(1, (1 << 27) // H)
        if op == "norm":
            out = {"y": torch.empty(R, H, **f64)}
            if case["residual"]:
                out["s"] = torch.empty(R, H, **f64)
            if case["e4m3"]:
                out["q"] = torch.empty(R, H, **f64)       # before the rounding to e4m3
                out["scale"] = torch.empty(R, **f64)
            for a in range(0, R, step):
                rows = slice(a, a + step)
                s = st["x"][rows].double()
                if case["residual"]:
                    s += st["r"][rows].double()
                    out["s"][rows] = s
                rms = (torch.linalg.vector_norm(s, dim=-1, keepdim=True) ** 2 / H + EPS).sqrt()
                y = out["y"][rows] = s / rms * w * on[rows]
                if case["e4m3"]:
                    big = y.abs().amax(-1)
                    scale = torch.where(big == 0, 1.0, big / 448)
                    out["scale"][rows] = scale
                    out["q"][rows] = y / scale[:, None]
            return out
        dx, dw = torch.empty(R, H, **f64), torch.zeros(H, **f64)
        for a in range(0, R, step):
            rows = slice(a, a + step)
            s, dy = st["s"][rows].double(), st["dy"][rows].double() * on[rows]
            rms = (torch.linalg.vector_norm(s, dim=-1, keepdim=True) ** 2 / H + EPS).sqrt()
            n = s / rms                          # y = n w, so dL/dn = dy w
            dn = dy * w
            dx[rows] = (dn - n * (dn * n).mean(-1, keepdim=True)) / rms
            if st["ds"] is not None:
                dx[rows] += st["ds"][rows].double()
            dw += (dy * n).sum(0)
        return {"dx": dx, "dw": dw}
    if op == "embed":
        out = torch.zeros(case["T"], H, **f64)
        real = st["ids"] >= 0
        out[real] = st["table"][st["ids"][real].long()].double() * st["scale"]
        return {"out": out}
    if op == "embed_bwd":
        dw = torch.zeros(case["V"], H, **f64)
        real = st["ids"] >= 0
        dw.index_add_(0, st["ids"][real].long(), st["dout"][real].double())
        return {"dw": dw.mul_(st["scale"])}
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2
                         for g in st["grads"]))
    c = min(1.0, case["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], dtype=torch.float64),
            "grads": [g.double() * c for g in st["grads"]]}
