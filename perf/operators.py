"""Operators around the MoE layer and the cases they are measured on.

op "decode": the whole layer for a few tokens (router, top-K, the selected experts' SwiGLU, weighted sum).
op "norm":   residual addition and root-mean-square norm in front of the router, forward and backward.
op "clip":   global norm of a list of gradients, and their scaling to at most a given norm.

run() computes them in plain torch operations, or, where `own` is true, through the framework's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of one request through a fine-grained layer: the latency of a decoding step
        {"name": "decode_1", "op": "decode", "dtype": "bf16", "N": 1, "H": 2048, "E": 64, "K": 6, "F": 1408},
        # a small batch of requests, most experts untouched or with one token
        {"name": "decode_8", "op": "decode", "dtype": "bf16", "N": 8, "H": 4096, "E": 64, "K": 4, "F": 2048},
        # a ragged batch that touches nearly every expert, several tokens for some
        {"name": "decode_33", "op": "decode", "dtype": "bf16", "N": 33, "H": 2048, "E": 64, "K": 6, "F": 1408},
        # few wide experts, a full decoding batch: many tokens for each
        {"name": "decode_64_wide", "op": "decode", "dtype": "bf16", "N": 64, "H": 4096, "E": 8, "K": 2, "F": 14336},
        # full precision, the smallest layer: launch latency only
        {"name": "decode_5_f32", "op": "decode", "dtype": "f32", "N": 5, "H": 128, "E": 4, "K": 2, "F": 256},
        # the norm of one decoded token
        {"name": "norm_1", "op": "norm", "dtype": "bf16", "N": 1, "H": 2048, "backward": False},
        # the norm of a training batch
        {"name": "norm_16384", "op": "norm", "dtype": "bf16", "N": 16384, "H": 4096, "backward": False},
        # its gradient, with the gradient that arrives through the residual stream
        {"name": "norm_16384_bwd", "op": "norm", "dtype": "bf16", "N": 16384, "H": 4096, "backward": True},
        # full precision, a ragged number of rows
        {"name": "norm_1021_f32_bwd", "op": "norm", "dtype": "f32", "N": 1021, "H": 7168, "backward": True},
        # the gradients of a small full-precision layer: launches only
        {"name": "clip_small", "op": "clip", "dtype": "f32", "E": 4, "H": 128, "F": 256, "copies": 2},
        # twelve layers' gradients of middling size, many tensors, odd lengths among them
        {"name": "clip_many", "op": "clip", "dtype": "mixed", "E": 8, "H": 1000, "F": 333, "copies": 12},
        # the gradients of one large layer
        {"name": "clip_large", "op": "clip", "dtype": "bf16", "E": 64, "H": 4096, "F": 2048, "copies": 1},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "norm", "norm", "clip"])
    if op == "decode":
        while True:
            dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
            E = _log_int(rng, 2, 256)
            c = {"op": op, "dtype": dtype, "N": _log_int(rng, 1, 64), "E": E, "K": rng.randint(1, min(8, E))}
            if dtype == "bf16":
                c.update(H=128 * _log_int(rng, 1, 56), F=128 * _log_int(rng, 1, 112))
            else:
                c.update(H=4 * _log_int(rng, 16, 512), F=_log_int(rng, 33, 1500))
            if E * c["H"] * c["F"] * (2 if dtype == "bf16" else 4) <= 8 * 4096 * 14336 * 2:
                return c
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        H = 8 * _log_int(rng, 16, 1024) if rng.random() < 0.5 else 128 * _log_int(rng, 1, 64)
        most = 16384 * 4096 * 2 // (H * (2 if dtype == "bf16" else 4))
        return {"op": op, "dtype": dtype, "N": _log_int(rng, 1, most), "H": H, "backward": rng.random() < 0.6}
    while True:
        c = {"op": op, "dtype": rng.choice(["bf16", "f32", "mixed"]), "E": _log_int(rng, 1, 64),
             "H": _log_int(rng, 16, 4096), "F": _log_int(rng, 16, 2048), "copies": _log_int(rng, 1, 12)}
        if c["copies"] * c["E"] * c["H"] * c["F"] * (2 if c["dtype"] == "bf16" else 4) <= 64 * 4096 * 2048 * 2:
            return c


def _gen(seed, k):
    return torch.Generator(device="cuda").manual_seed((int(seed) * 16 + k) % (1 << 62))


def _normal(shape, std, seed, k, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=_gen(seed, k))


def _clip_shapes(c):
    """A layer's gradients (router, experts, norm weight), `copies` layers; "mixed" alternates the types by tensor."""
    one = [(c["H"], c["E"]), (c["E"], c["H"], c["F"]), (c["E"], c["H"], c["F"]), (c["E"], c["F"], c["H"]), (c["H"],)]
    shapes = one * c["copies"]
    kinds = ["f32", "bf16"] if c["dtype"] == "mixed" else [c["dtype"]]
    return [(s, kinds[i % len(kinds)]) for i, s in enumerate(shapes)]


def prepare(case, seed):
    c = case
    if c["op"] == "clip":
        grads = [_normal(s, 1e-3, seed, i, DTYPES[d]) for i, (s, d) in enumerate(_clip_shapes(c))]
        # a user's limit: two fifths of the norm of such gradients, so the scaling happens
        total = sum(g.numel() for g in grads)
        state = {"case": c, "grads": grads, "max_norm": 0.4e-3 * math.sqrt(total),
                 "outs": [torch.empty_like(g) for g in grads]}
        if own:
            import dropless_top_moe_b200 as moe
            state["ws"] = moe.clip_workspace(grads)
        return state
    dtype, N, H = DTYPES[c["dtype"]], c["N"], c["H"]
    if c["op"] == "norm":
        weight = _normal((H,), 0.1, seed, 0, torch.float32).add_(1.0).to(dtype)
        state = {"case": c, "weight": weight}
        for k, name in enumerate(("dy", "h", "dh") if c["backward"] else ("x", "residual")):
            state[name] = _normal((N, H), 1.0, seed, 1 + k, dtype)
        return state
    E, K, F = c["E"], c["K"], c["F"]
    state = {"case": c,
             "W_r": _normal((H, E), 0.02, seed, 1, dtype),
             "W1": _normal((E, H, F), H ** -0.5, seed, 2, dtype),
             "W3": _normal((E, H, F), H ** -0.5, seed, 3, dtype),
             "W2": _normal((E, F, H), F ** -0.5, seed, 4, dtype)}
    # tokens whose K+1 largest logits are apart, so that the order of the sums does not decide the routing
    x = _normal((2 * N + 64, H), 1.0, seed, 0, dtype)
    logits = x.double() @ state["W_r"].double()
    top = logits.topk(min(K + 1, E), dim=1).values
    near = (top[:, :-1] - top[:, 1:]).amin(dim=1) < 1e-4 if top.shape[1] > 1 else torch.zeros_like(top[:, 0], dtype=torch.bool)
    state["x"] = x[torch.sort(near.to(torch.int32), stable=True).indices[:N]].contiguous()
    if own:
        import dropless_top_moe_b200 as moe
        state["layer"] = moe.MoEDecodeLayer(N, H, E, K, F, dtype=dtype)
    return state


def _route(logits, K):
    """K largest logits by column order among equals, and their softmax."""
    values, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    kept = torch.exp(values[:, :K] - values[:, :1])
    return ids[:, :K], kept / kept.sum(dim=1, keepdim=True)


def _decode_plain(s):
    c, x = s["case"], s["x"]
    N, E, K = c["N"], c["E"], c["K"]
    ids, w = _route(x.double() @ s["W_r"].double(), K)   # in 64 bits: which experts are kept hangs on it
    w = w.float()
    if 2 * N * K <= E:   # few assignments: fetch each one's expert
        flat = ids.reshape(-1)
        xs = x.float().repeat_interleave(K, dim=0).unsqueeze(1)
        g = torch.bmm(xs, s["W1"][flat].float())
        u = torch.bmm(xs, s["W3"][flat].float())
        out = torch.bmm(g / (1 + torch.exp(-g)) * u, s["W2"][flat].float()).view(N, K, -1)
        y = (w.unsqueeze(2) * out).sum(dim=1)
    else:                # every expert on every token, those not selected with weight zero
        xs = x.float().unsqueeze(0).expand(E, -1, -1)
        g = torch.bmm(xs, s["W1"].float())
        u = torch.bmm(xs, s["W3"].float())
        full = torch.zeros(N, E, device=x.device).scatter_(1, ids, w)
        out = torch.bmm(g / (1 + torch.exp(-g)) * u * full.t().unsqueeze(2), s["W2"].float())
        y = out.sum(dim=0)
    return {"y": y.to(x.dtype), "top_experts": ids.to(torch.int32), "weights": w}


def _norm_plain(s):
    weight = s["weight"].float()
    if not s["case"]["backward"]:
        h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)   # the residual stream as it is kept
        hf = h.float()
        rstd = torch.rsqrt((hf * hf).mean(dim=1, keepdim=True) + EPS)
        return {"y": (hf * rstd * weight).to(h.dtype), "h": h}
    dy, hf = s["dy"].float(), s["h"].float()
    rstd = torch.rsqrt((hf * hf).mean(dim=1, keepdim=True) + EPS)
    xhat = hf * rstd
    g = dy * weight
    dx = rstd * (g - xhat * (g * xhat).mean(dim=1, keepdim=True)) + s["dh"].float()
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * xhat).sum(dim=0).to(s["dy"].dtype)}


def _clip_plain(s):
    squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]])
    norm = squares.sum().sqrt().float()
    factor = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm.reshape(1), "grads": [(g.float() * factor).to(g.dtype) for g in s["grads"]]}


def _run_own(s):
    import dropless_top_moe_b200 as moe
    op = s["case"]["op"]
    if op == "decode":
        layer = s["layer"]
        y = layer.forward(s["x"], s["W_r"], s["W1"], s["W3"], s["W2"])
        return {"y": y, "top_experts": layer.top_experts, "weights": layer.weights}
    if op == "norm":
        if s["case"]["backward"]:
            dx, dweight = moe.moe_add_rms_norm_bwd(s["dy"], s["h"], s["weight"], dh=s["dh"], eps=EPS)
            return {"dx": dx, "dweight": dweight}
        y, h = moe.moe_add_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        return {"y": y, "h": h}
    norm = moe.moe_clip_grad_norm(s["grads"], s["max_norm"], outs=s["outs"], ws=s["ws"])
    return {"norm": norm, "grads": s["outs"]}


def run(state):
    if own:
        return _run_own(state)
    return {"decode": _decode_plain, "norm": _norm_plain, "clip": _clip_plain}[state["case"]["op"]](state)


def work(case):
    c = case
    if c["op"] == "clip":
        n = [(math.prod(s), 4 if d == "f32" else 2) for s, d in _clip_shapes(c)]
        return {"bytes": sum(2 * k * b for k, b in n), "flops": sum(3 * k for k, _ in n)}
    eb = 2 if c["dtype"] == "bf16" else 4
    N, H = c["N"], c["H"]
    if c["op"] == "norm":
        rows = 4 * N * H * eb   # two read and two written, or three read and one written
        return {"bytes": rows + (2 if c["backward"] else 1) * H * eb, "flops": (11 if c["backward"] else 5) * N * H}
    E, K, F = c["E"], c["K"], c["F"]
    used = E * (1.0 - (1.0 - K / E) ** N)   # distinct experts of N independent tokens
    return {"bytes": (H * E + used * 3 * H * F + 2 * N * H) * eb + 8 * N * K,
            "flops": 2 * N * H * E + 6 * N * K * H * F}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "clip":
        total = 0.0
        for g in s["grads"]:
            for part in g.reshape(-1).split(1 << 26):
                p = part.double()
                total += float((p * p).sum())
        norm = math.sqrt(total)
        factor = min(1.0, s["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
                "grads": [g.double().mul_(factor) for g in s["grads"]]}
    if c["op"] == "norm":
        N, H = c["N"], c["H"]
        w = s["weight"].double()
        if not c["backward"]:
            h = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
            scale = 1.0 / torch.sqrt(torch.einsum("nh,nh->n", h, h) / H + EPS)
            return {"y": torch.einsum("nh,n,h->nh", h, scale, w), "h": h}
        h, dy = s["h"].double(), s["dy"].double()
        scale = 1.0 / torch.sqrt(torch.einsum("nh,nh->n", h, h) / H + EPS)
        dot = torch.einsum("nh,nh,h->n", dy, h, w) * scale ** 3 / H
        dx = dy * w * scale[:, None] - h * dot[:, None] + s["dh"].double()
        return {"dx": dx, "dweight": torch.einsum("nh,nh,n->h", dy, h, scale)}
    N, E, K = c["N"], c["E"], c["K"]
    x = s["x"].double()
    logits = torch.einsum("nh,he->ne", x, s["W_r"].double())
    left = logits.clone()
    ids = torch.zeros(N, K, dtype=torch.int64, device="cuda")
    for k in range(K):
        ids[:, k] = torch.argmax(left, dim=1)
        left.scatter_(1, ids[:, k:k + 1], -math.inf)
    p = torch.softmax(logits, dim=1).gather(1, ids)
    w = p / p.sum(dim=1, keepdim=True)
    y = torch.zeros(N, c["H"], dtype=torch.float64, device="cuda")
    for e in torch.unique(ids).tolist():
        n, k = torch.nonzero(ids == e, as_tuple=True)
        g = x[n] @ s["W1"][e].double()
        a = g * torch.sigmoid(g) * (x[n] @ s["W3"][e].double())
        y.index_add_(0, n, (a @ s["W2"][e].double()) * w[n, k].unsqueeze(1))
    return {"y": y, "top_experts": ids.to(torch.int32), "weights": w}
