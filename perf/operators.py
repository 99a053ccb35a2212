"""Cases for measuring the library's matrix-optimizer and expert-routing operators.

Four operators:

  ortho      slide_orthogonalize: the Newton-Schulz orthogonal factor of a batch of matrices (the core of Muon)
  muon       slide_muon_step: mean of R gradient replicas, momentum, orthogonal factor, decoupled decay,
             FP32 master and BF16 copy
  route      slide_route_experts: scores, bias for balance, groups, top-k, renormalised weights, load; with
             "balance" followed by slide_route_bias_step, as once per training step
  route_bwd  slide_route_experts_backward: the gradient of the routing weights with respect to the logits

`own` False computes them in elementary torch operations in 32 bits; `own` True calls the library.
"""
import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)  # the quintic of every Newton-Schulz step
STEPS = 5
EPS = 1e-7
LR, MOMENTUM, DECAY = 1e-5, 0.95, 0.01
RATE = 1e-3                         # step of the balancing bias
TINY = 1e-20                        # added to the sum that renormalised weights are divided by
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the 64 x 2560 gate of a small router: the smallest matrix a step meets, all latency
        {"name": "ortho router gate", "op": "ortho", "batch": 1, "rows": 64, "cols": 2560, "type": "fp32"},
        # key and value projections of an h=2560 layer, as they lie (input size first): tall
        {"name": "ortho h2560 k,v", "op": "ortho", "batch": 2, "rows": 2560, "cols": 1024, "type": "bf16"},
        # one expert layer's down projections: many equal small matrices, ragged
        {"name": "ortho 40 experts", "op": "ortho", "batch": 40, "rows": 1000, "cols": 2187, "type": "bf16"},
        # the largest matrix of an h=5120 layer, from the FP32 momentum
        {"name": "ortho h5120 gate", "op": "ortho", "batch": 1, "rows": 5120, "cols": 17408, "type": "fp32"},
        # whole steps: the attention output of an h=2560 layer, one replica
        {"name": "muon h2560 o", "op": "muon", "batch": 1, "rows": 4096, "cols": 2560, "replicas": 1, "type": "bf16"},
        # ragged expert matrices with FP32-accumulated gradients of two replicas
        {"name": "muon 7 odd experts", "op": "muon", "batch": 7, "rows": 1001, "cols": 2731, "replicas": 2, "type": "fp32"},
        # gate and up projections of an h=2560 layer, four replicas
        {"name": "muon h2560 gate,up", "op": "muon", "batch": 2, "rows": 2560, "cols": 9728, "replicas": 4, "type": "bf16"},
        # single tokens while serving: nothing but latency
        {"name": "route 1 token", "op": "route", "tokens": 1, "experts": 256, "top_k": 8, "score": "sigmoid", "groups": 8,
         "top_groups": 4, "bias": True, "mask": False, "renorm": True, "balance": False, "type": "fp32"},
        # an odd prompt through a softmax router without groups, BF16 logits
        {"name": "route softmax 4099", "op": "route", "tokens": 4099, "experts": 60, "top_k": 4, "score": "softmax", "groups": 1,
         "top_groups": 1, "bias": False, "mask": False, "renorm": False, "balance": False, "type": "bf16"},
        # a training step's tokens with padding, load counted and the bias moved
        {"name": "route train 65536", "op": "route", "tokens": 65536, "experts": 256, "top_k": 8, "score": "sigmoid", "groups": 8,
         "top_groups": 4, "bias": True, "mask": True, "renorm": True, "balance": True, "type": "fp32"},
        # gradients of the same, and of a softmax router that does not renormalise
        {"name": "route_bwd sigmoid 65536", "op": "route_bwd", "tokens": 65536, "experts": 256, "top_k": 8, "score": "sigmoid",
         "groups": 1, "top_groups": 1, "bias": False, "mask": True, "renorm": True, "type": "fp32"},
        {"name": "route_bwd softmax 8191", "op": "route_bwd", "tokens": 8191, "experts": 60, "top_k": 4, "score": "softmax",
         "groups": 1, "top_groups": 1, "bias": False, "mask": False, "renorm": False, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("ortho", "muon", "route", "route_bwd"))
    if op in ("ortho", "muon"):
        while True:
            rows, cols, batch = _log(rng, 16, 8192), _log(rng, 16, 17408), _log(rng, 1, 64)
            if rng.random() < 0.5:  # sizes of real layers are mostly multiples of 64
                rows, cols = max(64, rows // 64 * 64), max(64, cols // 64 * 64)
            m, n = min(rows, cols), max(rows, cols)
            if batch * m * m * (3 * n + m) <= 1.2e12 and batch * m * n <= 9e7:
                break
        c = {"op": op, "batch": batch, "rows": rows, "cols": cols, "type": rng.choice(("bf16", "fp32"))}
        if op == "muon":
            c["replicas"] = rng.randint(1, 4)
        return c
    groups = rng.choice((1, 1, 4, 8))
    experts = groups * rng.randint(max(2, 8 // groups), 512 // groups)
    if groups > 1:
        score, bias, top_groups = "sigmoid", rng.random() < 0.7, rng.randint(2, groups)
    else:
        score, bias, top_groups = rng.choice(("sigmoid", "softmax")), False, 1
        bias = score == "sigmoid" and rng.random() < 0.5
    top_k = rng.randint(1, min(12, experts // groups * top_groups))
    c = {"op": op, "tokens": _log(rng, 1, 65536), "experts": experts, "top_k": top_k, "score": score, "groups": groups,
         "top_groups": top_groups, "bias": bias, "mask": rng.random() < 0.3, "renorm": rng.random() < 0.6,
         "type": rng.choice(("bf16", "fp32"))}
    while c["tokens"] * c["experts"] > 65536 * 256:
        c["tokens"] //= 2
    if op == "route":
        c["balance"] = bias and rng.random() < 0.5
    return c


def _spectrum(g, batch, rows, cols, rms):
    """Matrices as gradients are: a few strong directions with falling weights over noise."""
    r = min(16, rows, cols)
    u = torch.randn(batch, rows, r, generator=g, device="cuda")
    v = torch.randn(batch, r, cols, generator=g, device="cuda")
    w = torch.arange(1, r + 1, device="cuda", dtype=torch.float32).rsqrt() * 0.3
    x = torch.randn(batch, rows, cols, generator=g, device="cuda")
    return x.baddbmm_(u * w, v).mul_(rms)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    s = dict(case, ws=None)
    dt = TYPES[case["type"]]
    if case["op"] == "ortho":
        s["x"] = _spectrum(g, case["batch"], case["rows"], case["cols"], 1e-3).to(dt)
        s["out"] = torch.empty(s["x"].shape, dtype=torch.bfloat16, device="cuda")
        return s
    if case["op"] == "muon":
        shape = (case["batch"], case["rows"], case["cols"])
        common = _spectrum(g, *shape, 1e-3)
        s["grads"] = [(common + torch.randn(shape, generator=g, device="cuda") * 1e-3).to(dt) for _ in range(case["replicas"])]
        s["momentum"] = _spectrum(g, *shape, 3e-4)
        s["master"] = torch.randn(shape, generator=g, device="cuda") * 0.02
        s["bf16"] = s["master"].bfloat16()
        return s
    T, E, K = case["tokens"], case["experts"], case["top_k"]
    # logits of a trained router: per-expert offsets over the tokens' own preferences
    x = torch.randn(T, E, generator=g, device="cuda") * 1.2 + torch.randn(E, generator=g, device="cuda") * 0.4 - 0.5
    s["mask"] = None
    if case["mask"]:  # padding tokens, whose logits hold anything
        s["mask"] = (torch.rand(T, generator=g, device="cuda") < 0.9).to(torch.uint8)
        x[s["mask"] == 0] = float("nan")
    s["logits"] = x.to(dt)
    s["bias"] = (torch.randint(-100, 101, (E,), generator=g, device="cuda").float() * RATE) if case["bias"] else None
    s["weights"] = torch.empty(T, K, device="cuda")
    s["chosen"] = torch.empty(T, K, dtype=torch.int32, device="cuda")
    if case["op"] == "route":
        s["load"] = torch.zeros(E, dtype=torch.int64, device="cuda")
        return s
    s["chosen"] = torch.sort(torch.where(torch.isnan(x), 0.0, x), dim=1, descending=True, stable=True)[1][:, :K].to(torch.int32).contiguous()
    if s["mask"] is not None:
        s["chosen"][s["mask"] == 0] = -1
    s["d_weights"] = torch.randn(T, K, generator=g, device="cuda")
    s["d_logits"] = torch.empty(T, E, dtype=dt, device="cuda")
    return s


# ---- the plain forms ---------------------------------------------------------


def _newton_schulz(x):
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / ((x * x).sum(dim=(-2, -1), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFS
    for _ in range(STEPS):
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.mT if tall else x


def _plain_muon(s):
    g = sum(r.float() for r in s["grads"]) / len(s["grads"])
    s["momentum"].mul_(MOMENTUM).add_(g * (1 - MOMENTUM))
    u = s["momentum"] * MOMENTUM + g * (1 - MOMENTUM)
    scale = 0.2 * math.sqrt(max(s["rows"], s["cols"]))
    s["master"].mul_(1 - LR * DECAY).sub_(_newton_schulz(u) * (LR * scale))
    s["bf16"].copy_(s["master"])
    return {"master": s["master"], "momentum": s["momentum"], "bf16": s["bf16"]}


def _scores(s, x):
    if s["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _plain_route(s):
    x = s["logits"].float()
    T, E, G, K = s["tokens"], s["experts"], s["groups"], s["top_k"]
    live = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    x = torch.where(live[:, None], x, 0.0)
    score = _scores(s, x)
    # the choice: by score plus bias; the softmax keeps the logits' order, so without a bias it is made on them
    key = x if s["score"] == "softmax" else score if s["bias"] is None else score + s["bias"]
    if G > 1:
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True)[0]
        rank = best[:, :, 0] + best[:, :, 1]
        kept = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, : s["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, kept, True)
        key = torch.where(keep.repeat_interleave(E // G, dim=1), key, -math.inf)
    chosen = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :K]
    w = score.gather(1, chosen)
    if s["renorm"]:
        w = w / (w.sum(dim=1, keepdim=True) + TINY)
    w = torch.where(live[:, None], w, 0.0)
    s["load"].index_add_(0, chosen.reshape(-1), live[:, None].expand(T, K).reshape(-1).to(torch.int64))
    out = {"weights": w, "experts": torch.where(live[:, None], chosen, -1).to(torch.int32)}
    if s["balance"]:
        load = s["load"]
        s["bias"].add_(torch.sign(load.sum() - load * E).float() * RATE)
        load.zero_()
        return dict(out, bias=s["bias"], load=load)
    return dict(out, load=s["load"])


def _plain_route_bwd(s):
    x, dw = s["logits"].float(), s["d_weights"]
    live = (s["chosen"] >= 0) if s["mask"] is None else (s["chosen"] >= 0) & (s["mask"] != 0)[:, None]
    at = torch.where(live, s["chosen"], 0).long()
    x = torch.where(live[:, :1], x, 0.0)
    score = _scores(s, x)
    p, dw = score.gather(1, at), torch.where(live, dw, 0.0)
    if s["renorm"]:
        total = p.sum(dim=1, keepdim=True) + TINY
        dp = (dw - (dw * p).sum(dim=1, keepdim=True) / total) / total
    else:
        dp = dw
    if s["score"] == "sigmoid":
        dx = torch.zeros_like(x).scatter_add_(1, at, torch.where(live, dp * p * (1.0 - p), 0.0))
    else:
        dx = torch.zeros_like(x).scatter_add_(1, at, torch.where(live, dp, 0.0))
        dx = score * (dx - (dp * p).sum(dim=1, keepdim=True)) if not s["renorm"] else score * dx
    return torch.where(live[:, :1], dx, 0.0).to(s["logits"].dtype)


# ---- one pass ------------------------------------------------------------------


def _own(s):
    import mixed_precision_adam_grad_gb300 as S
    stream = torch.cuda.current_stream()
    if s["op"] in ("ortho", "muon"):
        shape = s["batch"], s["rows"], s["cols"]
        if s["ws"] is None:  # a program allocates its workspace once
            s["ws"] = torch.empty(S.slide_ortho_workspace(*shape), dtype=torch.uint8, device="cuda")
        kind = S.SLIDE_TYPE_FP32 if s["type"] == "fp32" else S.SLIDE_TYPE_BF16
        if s["op"] == "ortho":
            S.slide_orthogonalize(*shape, s["x"], s["out"], S.ortho_params(steps=STEPS, eps=EPS), s["ws"], x_type=kind,
                                  stream=stream)
            return s["out"]
        hp = S.muon_hparams(lr=LR, momentum=MOMENTUM, weight_decay=DECAY, steps=STEPS, eps=EPS)
        S.slide_muon_step(*shape, s["grads"], s["master"], s["momentum"], s["bf16"], hp, s["ws"], grads_type=kind, stream=stream)
        return {"master": s["master"], "momentum": s["momentum"], "bf16": s["bf16"]}
    cfg = S.route_config(s["experts"], s["top_k"], score=S.SLIDE_SCORE_SIGMOID if s["score"] == "sigmoid" else S.SLIDE_SCORE_SOFTMAX,
                         n_groups=s["groups"], top_groups=s["top_groups"], renormalize=s["renorm"])
    kind = S.SLIDE_TYPE_FP32 if s["type"] == "fp32" else S.SLIDE_TYPE_BF16
    if s["op"] == "route_bwd":
        S.slide_route_experts_backward(s["tokens"], s["logits"], s["chosen"], s["d_weights"], s["d_logits"], cfg,
                                       token_mask=s["mask"], logits_type=kind, stream=stream)
        return s["d_logits"]
    S.slide_route_experts(s["tokens"], s["logits"], s["weights"], s["chosen"], cfg, bias=s["bias"], token_mask=s["mask"],
                          load=s["load"], logits_type=kind, stream=stream)
    out = {"weights": s["weights"], "experts": s["chosen"], "load": s["load"]}
    if s["balance"]:
        S.slide_route_bias_step(s["experts"], s["load"], s["bias"], RATE, stream=stream)
        out["bias"] = s["bias"]
    return out


def run(state):
    if own:
        return _own(state)
    if state["op"] == "ortho":
        return _newton_schulz(state["x"].float()).bfloat16()
    return {"muon": _plain_muon, "route": _plain_route, "route_bwd": _plain_route_bwd}[state["op"]](state)


def work(case):
    size = {"bf16": 2, "fp32": 4}[case["type"]]
    if case["op"] in ("ortho", "muon"):
        m, n = min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        r = n / m
        # symmetric products count half; the iteration on the matrix, or on its Gram matrix where that is less
        flops = case["batch"] * m ** 3 * min(STEPS * (3 * r + 1), 3 * r + 4 * STEPS - 3)
        each = size + 2 if case["op"] == "ortho" else case["replicas"] * size + 18
        return {"bytes": case["batch"] * m * n * each, "flops": flops}
    T, E, K = case["tokens"], case["experts"], case["top_k"]
    if case["op"] == "route":
        return {"bytes": T * (E * size + K * 8 + case["mask"]) + 8 * E + 4 * E * case["bias"], "flops": 6.0 * T * E}
    # a gradient that only the chosen experts have needs their logits alone
    read = E if case["score"] == "softmax" and not case["renorm"] else K
    return {"bytes": T * (read * size + K * 8 + E * size + case["mask"]), "flops": 6.0 * T * (read + K)}


# ---- the definitions in 64 bits ------------------------------------------------


def _polar_poly(u, steps):
    """The Newton-Schulz polynomial of u / (|u| + eps), applied by its odd powers."""
    u = u.double()
    norm = torch.linalg.vector_norm(u, dim=(1, 2), keepdim=True)
    x = u / (norm + EPS)
    a, b, c = COEFFS
    left = x.shape[1] <= x.shape[2]
    eye = torch.eye(min(x.shape[1], x.shape[2]), dtype=torch.float64, device=x.device)
    done = 0
    while done < steps:
        q = torch.bmm(x, x.transpose(1, 2)) if left else torch.bmm(x.transpose(1, 2), x)
        poly = a * eye + torch.bmm(q, b * eye + c * q)
        x = torch.bmm(poly, x) if left else torch.bmm(x, poly)
        done += 1
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ortho":
        return _polar_poly(s["x"], STEPS)
    if case["op"] == "muon":
        g = torch.stack([r.double() for r in s["grads"]]).mean(dim=0)
        mom = MOMENTUM * s["momentum"].double() + (1 - MOMENTUM) * g
        o = _polar_poly(MOMENTUM * mom + (1 - MOMENTUM) * g, STEPS)
        scale = 0.2 * max(case["rows"], case["cols"]) ** 0.5
        th = s["master"].double() * (1 - LR * DECAY) - LR * scale * o
        return {"master": th, "momentum": mom, "bf16": th}
    x = s["logits"].double()
    on = torch.ones(case["tokens"], 1, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"].bool().unsqueeze(1)
    x = x.masked_fill(~on, 0.0)
    p = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, dim=1)
    if case["op"] == "route":
        # the choice itself is defined on FP32 scores, so that near ties are decided the same way everywhere
        x32 = x.float()
        key = x32 if case["score"] == "softmax" else (x32.neg().exp() + 1).reciprocal()
        if s["bias"] is not None:
            key = key + s["bias"]
        T, E, G = case["tokens"], case["experts"], case["groups"]
        if G > 1:
            per = key.unflatten(1, (G, E // G))
            rank = per.topk(2, dim=2).values.sum(dim=2)
            order = rank.argsort(dim=1, descending=True, stable=True)
            place = order.argsort(dim=1)
            key = per.masked_fill((place >= case["top_groups"]).unsqueeze(2), -math.inf).flatten(1)
        chosen = key.argsort(dim=1, descending=True, stable=True)[:, : case["top_k"]]
        w = torch.take_along_dim(p, chosen, dim=1)
        if case["renorm"]:
            w = w / (w.sum(dim=1, keepdim=True) + TINY)
        out = {"weights": w.masked_fill(~on, 0.0), "experts": None, "load": None}
        if case["balance"]:
            load = torch.bincount(chosen[on[:, 0]].reshape(-1), minlength=E).double()
            out["bias"] = s["bias"].double() + RATE * torch.sign(load.mean() - load)
        return out
    pick = torch.zeros_like(x)
    at = s["chosen"].long().clamp(min=0)
    pick.scatter_(1, at, s["d_weights"].double() * (s["chosen"] >= 0))
    hit = torch.zeros_like(x).scatter_(1, at, (s["chosen"] >= 0).double())
    if case["renorm"]:
        total = (p * hit).sum(dim=1, keepdim=True) + TINY
        w = p * hit / total
        dp = hit * (pick - (pick * w).sum(dim=1, keepdim=True)) / total
    else:
        dp = pick
    if case["score"] == "sigmoid":
        dx = dp * p * (1 - p)
    else:
        dx = p * (dp - (dp * p).sum(dim=1, keepdim=True))
    return dx.masked_fill(~on, 0.0)
