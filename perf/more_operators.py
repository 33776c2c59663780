"""The operators around the expert MLP in a block of a model, as they are
measured: the residual addition with the root-mean-square norm that feeds the
layer (bf16 and MXFP8) and its backward pass, routing by softmax or sigmoid
scores with a selection bias and expert groups and its backward pass, and the
norm over all gradients with clipping.

Each case is one pass through one operator.  `run` computes it in plain torch
operations, or, where `own` is true, through the framework's entry points.
Sizes are those of the framework's layers (tiny: 256 tokens, H = 128, I = 256,
4 experts top-2; Mixtral: 16384 tokens, H = 4096, I = 14336, 8 experts top-2;
fine-grained: 8192 tokens, H = 2048, I = 1024, 64 experts top-8; up to 256
experts), and odd ones between them.
"""
import math

import torch

own = False

EPS = 1e-6            # under the root of the norm
MAX_NORM = 1.0        # of the clipped gradients


def listed():
    return [
        # one token of a decoder: the norm before the layer, its codes for the expert GEMMs (latency)
        {"name": "norm_fwd_1x4096", "op": "norm_fwd", "T": 1, "H": 4096, "residual": "bf16", "w32": False,
         "codes": True},
        # the Mixtral layer's tokens: residual stream, bf16 for router and training, codes for the expert GEMMs
        {"name": "norm_fwd_16384x4096", "op": "norm_fwd", "T": 16384, "H": 4096, "residual": "bf16", "w32": False,
         "codes": True},
        # an odd number of tokens of an odd width with an fp32 residual stream
        {"name": "norm_fwd_5003x1000", "op": "norm_fwd", "T": 5003, "H": 1000, "residual": "f32", "w32": True,
         "codes": False},
        # the Mixtral layer's backward, the residual stream's gradient joined
        {"name": "norm_bwd_16384x4096", "op": "norm_bwd", "T": 16384, "H": 4096, "residual": "bf16", "w32": False},
        # the tiny layer's backward without a residual stream (latency)
        {"name": "norm_bwd_256x128", "op": "norm_bwd", "T": 256, "H": 128, "residual": None, "w32": True},
        # a ragged handful of decoder tokens: sigmoid scores, bias, groups (latency)
        {"name": "route_fwd_7x256", "op": "route_fwd", "T": 7, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5},
        # the same router on a long batch
        {"name": "route_fwd_65536x256", "op": "route_fwd", "T": 65536, "E": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5},
        # the fine-grained layer with softmax weights as they are, an odd number of tokens
        {"name": "route_fwd_8191x64", "op": "route_fwd", "T": 8191, "E": 64, "k": 8, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_top": 1, "renorm": False, "scale": 1.0},
        # its gradient, dense because the softmax is not renormalised, beside the balance loss's
        {"name": "route_bwd_8191x64", "op": "route_bwd", "T": 8191, "E": 64, "k": 8, "score": "softmax",
         "renorm": False, "scale": 1.0, "add": True},
        # the gradient of the sigmoid router on the long batch
        {"name": "route_bwd_65536x256", "op": "route_bwd", "T": 65536, "E": 256, "k": 8, "score": "sigmoid",
         "renorm": True, "scale": 2.5, "add": False},
        # the tiny layer's gradients: norm weight, router, both expert weights (latency)
        {"name": "clip_tiny", "op": "clip", "layers": 1, "H": 128, "I": 256, "E": 4, "main32": False, "odd": 0},
        # two fine-grained layers from their fp32 accumulators, and odd vectors beside them
        {"name": "clip_fine", "op": "clip", "layers": 2, "H": 2048, "I": 1024, "E": 64, "main32": True, "odd": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "route_fwd", "route_bwd", "clip"])
    if op in ("norm_fwd", "norm_bwd"):
        while True:
            c = {"op": op, "T": _log(rng, 1, 65536), "H": 8 * _log(rng, 8, 2048),
                 "residual": rng.choice([None, "bf16", "f32"]), "w32": rng.random() < 0.5}
            if op == "norm_fwd":
                c["codes"] = rng.random() < 0.5
                if c["codes"]:
                    c["H"] = 128 * _log(rng, 1, 128)
            if c["T"] * c["H"] <= 16384 * 4096 * (0.5 if c["residual"] == "f32" else 1):
                return c
    if op in ("route_fwd", "route_bwd"):
        E = _log(rng, 2, 256)
        c = {"op": op, "T": _log(rng, 1, 65536), "E": E, "k": rng.randint(1, min(8, E)),
             "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.5,
             "scale": rng.choice([1.0, 2.5])}
        if op == "route_bwd":
            c["add"] = rng.random() < 0.5
            c["renorm"] = c["renorm"] and c["k"] > 1                   # one renormalised weight has no gradient
            return c
        c["bias"] = rng.random() < 0.5
        c["groups"] = rng.choice([g for g in range(1, min(E, 32) + 1) if E % g == 0])
        size = E // c["groups"]
        c["top_groups"] = rng.randint(-(-c["k"] // size), c["groups"])
        c["group_top"] = rng.randint(1, 2) if size > 1 else 1
        return c
    top = _elements({"layers": 2, "H": 2048, "I": 1024, "E": 64, "odd": 8})
    while True:
        c = {"op": "clip", "layers": rng.randint(1, 8), "H": 8 * _log(rng, 8, 512), "I": 8 * _log(rng, 8, 1024),
             "E": _log(rng, 1, 64), "main32": rng.random() < 0.5, "odd": rng.randint(0, 16)}
        if _elements(c) <= top:
            return c


def _shapes(c):
    """The gradients of a block's layers: norm weight, router, both expert weights, and odd vectors (a head's, a bias's)."""
    H, I, E = c["H"], c["I"], c["E"]
    layer = [((H,), True), ((E, H), True), ((E, 2 * I, H), c.get("main32", True)), ((E, H, I), c.get("main32", True))]
    return layer * c["layers"] + [((1 + 997 * i * i,), i % 2 == 0) for i in range(c["odd"])]


def _elements(c):
    return sum(math.prod(shape) for shape, _ in _shapes(c))


def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        T, H = case["T"], case["H"]
        stream = {None: 0, "bf16": 2, "f32": 4}[case["residual"]]
        w = (4 if case["w32"] else 2) * H
        if op == "norm_fwd":
            n = T * H * (2 + 2 * stream + 2) + 4 * T + w
            return {"bytes": n + (T * H + T * H // 32 if case["codes"] else 0), "flops": 5 * T * H}
        r = 4 if case["residual"] == "f32" else 2
        return {"bytes": T * H * (2 + r + stream + 2 + (4 if case["residual"] == "f32" else 0)) + 4 * T + w + 4 * H,
                "flops": 10 * T * H}
    if op == "route_fwd":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 6 * T * E}
    if op == "route_bwd":
        T, E, k = case["T"], case["E"], case["k"]
        dense = case["score"] == "softmax" and not case["renorm"]
        chosen = 4 * T * k if case["score"] == "sigmoid" else 0        # the chosen logits
        return {"bytes": 4 * T * E * (1 + dense + case["add"]) + 12 * T * k + chosen, "flops": 4 * T * E}
    n = sum(math.prod(shape) * (4 if f32 else 2) for shape, f32 in _shapes(case))
    return {"bytes": 2 * n + 4, "flops": 3 * _elements(case)}


# ------------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    op = case["op"]
    s = {"case": case}
    if op in ("norm_fwd", "norm_bwd"):
        T, H = case["T"], case["H"]
        column = 1.0 + 20.0 * (torch.rand(H, generator=g, device="cuda") < 0.01)       # a few loud channels
        weight = 1.0 + normal(H, std=0.1)
        s["weight"] = weight if case["w32"] else weight.bfloat16()
        stream = torch.float32 if case["residual"] == "f32" else torch.bfloat16
        if op == "norm_fwd":
            s["x"] = normal(T, H).bfloat16()
            s["residual"] = None if case["residual"] is None else (normal(T, H, std=3.0) * column).to(stream)
            s["residual_out"] = None if case["residual"] is None else torch.empty((T, H), dtype=stream, device="cuda")
            s["y"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
            s["rstd"] = torch.empty(T, device="cuda")
            s["q"] = torch.empty((T, H), dtype=torch.uint8, device="cuda") if case["codes"] else None
            s["s"] = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda") if case["codes"] else None
            return s
        r = normal(T, H, std=3.0) * column
        s["rstd"] = torch.rsqrt(r.square().mean(dim=1) + EPS)
        s["r"] = r.to(stream)
        s["dy"] = normal(T, H, std=1e-3).bfloat16()
        s["dresidual"] = None if case["residual"] is None else normal(T, H, std=1e-3).to(stream)
        s["dx"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        s["dresidual_out"] = torch.empty((T, H), device="cuda") if case["residual"] == "f32" else None
        s["dweight"] = torch.empty(H, device="cuda")
        return s
    if op in ("route_fwd", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = (normal(T, E, std=1.5) + normal(1, E)).contiguous()              # some experts are preferred
        if op == "route_fwd":
            s["bias"] = normal(E, std=0.05) if case["bias"] else None
            s["ids"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
            s["probs"] = torch.empty((T, k), device="cuda")
            return s
        score = _scores(s["logits"], case["score"])
        top = torch.topk(score, k, dim=1)
        p = top.values / top.values.sum(dim=1, keepdim=True) if case["renorm"] else top.values
        s["ids"] = top.indices.to(torch.int32).contiguous()
        s["probs"] = (p * case["scale"]).float().contiguous()
        s["dprobs"] = normal(T, k, std=1e-2)
        s["dlogits_in"] = normal(T, E, std=1e-4) if case["add"] else None              # the balance loss's part
        s["dlogits"] = torch.empty((T, E), device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    # gradients of sizes that differ by layer and kind, as a step leaves them; an expert without tokens has zeros
    grads = []
    for i, (shape, f32) in enumerate(_shapes(case)):
        t = normal(*shape, std=10.0 ** (-3 + (i % 3)))
        if len(shape) == 3 and shape[0] > 2:
            t[1] = 0.0
        grads.append(t if f32 else t.bfloat16())
    s["grads"] = grads
    s["out"] = [torch.empty_like(t) for t in grads]
    return s


# --------------------------------------------------------------- plain forms --

def _plain_norm_fwd(s):
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    rstd = 1.0 / torch.sqrt((r * r).mean(dim=1) + EPS)
    y = (r * rstd[:, None] * s["weight"].float()).bfloat16()
    out = {"y": y, "rstd": rstd}
    if s["residual"] is not None:
        out["residual"] = r.to(s["residual"].dtype)
    if s["q"] is not None:
        T, H = y.shape
        blocks = y.float().reshape(T, H // 32, 32)
        # floor(log2) of the largest magnitude - 8, at least -127
        exponent = (torch.frexp(blocks.abs().amax(dim=2)).exponent - 9).clamp(min=-127)
        codes = torch.ldexp(blocks, -exponent[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        out["q"] = codes.reshape(T, H)
        out["s"] = (exponent + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _plain_norm_bwd(s):
    xh = s["r"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["weight"].float()
    d = s["rstd"][:, None] * (g - xh * (g * xh).mean(dim=1, keepdim=True))
    if s["dresidual"] is not None:
        d = d + s["dresidual"].float()
    out = {"dx": d.bfloat16(), "dweight": (dy * xh).sum(dim=0)}
    if s["dresidual_out"] is not None:
        out["dresidual"] = d
    return out


def _scores(z, kind):
    """In 64 bits: the choice of experts goes by differences that 32 bits lose."""
    z = z.double()
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    e = torch.exp(z - z.max(dim=1, keepdim=True).values)
    return e / e.sum(dim=1, keepdim=True)


def _plain_route_fwd(s):
    c = s["case"]
    T, E = s["logits"].shape
    score = _scores(s["logits"], c["score"])
    choice = score if s["bias"] is None else score + s["bias"].double()
    if c["top_groups"] < c["groups"]:
        size = E // c["groups"]
        best = choice.reshape(T, c["groups"], size).sort(dim=2, descending=True).values[:, :, :c["group_top"]].sum(dim=2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros_like(best).scatter(1, kept, 1.0).repeat_interleave(size, dim=1)
        choice = torch.where(keep > 0, choice, torch.full_like(choice, -math.inf))
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    p = score.gather(1, ids)
    if c["renorm"]:
        p = p / p.sum(dim=1, keepdim=True)
    return {"ids": ids.to(torch.int32), "probs": (p * c["scale"]).float()}


def _plain_route_bwd(s):
    c = s["case"]
    ids, p, dp = s["ids"].long(), s["probs"], s["dprobs"]
    z = s["logits"]
    total = (p * dp).sum(dim=1, keepdim=True)
    d = p * (dp - total / c["scale"]) if c["renorm"] else p * dp
    if c["score"] == "sigmoid":
        d = d / (1.0 + torch.exp(z.gather(1, ids)))                    # 1 - sigmoid
    base = torch.zeros_like(z)
    if c["score"] == "softmax" and not c["renorm"]:
        e = torch.exp(z - z.max(dim=1, keepdim=True).values)
        base = -(e / e.sum(dim=1, keepdim=True)) * total
    if s["dlogits_in"] is not None:
        base = base + s["dlogits_in"]
    return base.scatter_add(1, ids, d)


def _plain_clip(s):
    squares = [g.double().square().sum() for g in s["grads"]]
    norm = torch.sqrt(torch.stack(squares).sum())
    coef = torch.where(norm > MAX_NORM, MAX_NORM / norm, torch.ones_like(norm)).float()
    return {"norm": norm.float().reshape(1), "grads": [(g.float() * coef).to(g.dtype) for g in s["grads"]]}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "route_fwd": _plain_route_fwd,
                "route_bwd": _plain_route_bwd, "clip": _plain_clip}[op](s)
    import mxfp8_grouped_gemm_gb300 as mxg
    if op == "norm_fwd":
        mxg.mxg_rms_norm_fwd(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["residual_out"], y=s["y"],
                             rstd=s["rstd"], q=s["q"], s=s["s"])
        out = {"y": s["y"], "rstd": s["rstd"]}
        if s["residual"] is not None:
            out["residual"] = s["residual_out"]
        if s["q"] is not None:
            out["q"], out["s"] = s["q"].view(torch.float8_e4m3fn), s["s"].view(torch.float8_e8m0fnu)
        return out
    if op == "norm_bwd":
        mxg.mxg_rms_norm_bwd(s["dy"], s["r"], s["weight"], s["rstd"], dresidual=s["dresidual"], dx=s["dx"],
                             dresidual_out=s["dresidual_out"], dweight=s["dweight"])
        out = {"dx": s["dx"], "dweight": s["dweight"]}
        if s["dresidual_out"] is not None:
            out["dresidual"] = s["dresidual_out"]
        return out
    if op == "route_fwd":
        mxg.mxg_route_scores_fwd(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                 top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renorm"],
                                 scale=c["scale"], ids=s["ids"], probs=s["probs"])
        return {"ids": s["ids"], "probs": s["probs"]}
    if op == "route_bwd":
        return mxg.mxg_route_scores_bwd(s["logits"], s["ids"], s["probs"], s["dprobs"], s["status"], score=c["score"],
                                        renormalize=c["renorm"], scale=c["scale"], dlogits_in=s["dlogits_in"],
                                        dlogits=s["dlogits"])
    norm, out = mxg.mxg_grad_clip(s["grads"], MAX_NORM, out=s["out"])
    return {"norm": norm, "grads": out}


# ------------------------------------------------------------------ 64 bits --

def exact(case, seed):
    s = prepare(case, seed)
    op, dd = case["op"], torch.float64
    if op == "norm_fwd":
        r = s["x"].to(dd)
        if s["residual"] is not None:
            r = torch.add(r, s["residual"].to(dd))
        rstd = torch.pow(torch.einsum("th,th->t", r, r) / case["H"] + EPS, -0.5)
        y = torch.einsum("th,t,h->th", r, rstd, s["weight"].to(dd))
        out = {"y": y, "rstd": rstd}
        if s["residual"] is not None:
            out["residual"] = r
        if case["codes"]:
            held = y.bfloat16().to(dd)                                 # the codes are those of the bf16 matrix
            top = held.unflatten(1, (-1, 32)).abs().max(dim=2).values
            scale = torch.exp2(torch.clamp(torch.frexp(top).exponent.to(dd) - 9.0, min=-127.0))
            out["q"] = held / scale.repeat_interleave(32, dim=1)
            out["s"] = scale
        return out
    if op == "norm_bwd":
        r, dy, k = s["r"].to(dd), s["dy"].to(dd), s["rstd"].to(dd)
        g = dy * s["weight"].to(dd)[None, :]
        along = torch.einsum("th,th->t", g, r) * k.pow(3) / case["H"]
        d = torch.einsum("th,t->th", g, k) - torch.einsum("th,t->th", r, along)
        if s["dresidual"] is not None:
            d = d + s["dresidual"].to(dd)
        out = {"dx": d, "dweight": torch.einsum("th,th,t->h", dy, r, k)}
        if s["dresidual_out"] is not None:
            out["dresidual"] = d
        return out
    if op in ("route_fwd", "route_bwd"):
        z = s["logits"].to(dd)
        score = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, dim=1)
        T, E = z.shape
        if op == "route_fwd":
            rank = score if s["bias"] is None else score + s["bias"].to(dd)[None, :]
            if case["top_groups"] < case["groups"]:
                by_group = rank.unflatten(1, (case["groups"], -1))
                value = torch.topk(by_group, case["group_top"], dim=2).values.sum(dim=2)
                worst = torch.topk(value, case["top_groups"], dim=1).values[:, -1:]
                rank = by_group.masked_fill((value < worst)[:, :, None], -math.inf).flatten(1)
            chosen = torch.topk(rank, case["k"], dim=1).indices
            w = torch.gather(score, 1, chosen)
            if case["renorm"]:
                w = torch.nn.functional.normalize(w, p=1.0, dim=1, eps=0.0)
            return {"ids": None, "probs": w * case["scale"]}
        # dz = (dw/dz)^T dp by the chain rule through the scores of all experts
        pick = torch.nn.functional.one_hot(s["ids"].long(), E).to(dd)
        p, dp = s["probs"].to(dd), s["dprobs"].to(dd)
        own_score = torch.einsum("tke,te->tk", pick, score)
        if case["renorm"]:
            total = own_score.sum(dim=1, keepdim=True)
            ds = (dp * case["scale"] - torch.einsum("tk,tk->t", dp, p)[:, None]) / total
            own_score = p * total / case["scale"]
        else:
            ds = dp * case["scale"]
            own_score = p / case["scale"]
        dense = torch.einsum("tk,tke->te", ds * own_score, pick)
        if case["score"] == "sigmoid":
            dense = dense * torch.sigmoid(-z)
        else:
            dense = dense - score * torch.einsum("tk,tk->t", ds, own_score)[:, None]
        return dense if s["dlogits_in"] is None else dense + s["dlogits_in"].to(dd)
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.flatten(), dtype=dd)) ** 2 for g in s["grads"]))
    coef = min(1.0, MAX_NORM / norm) if norm else 1.0
    return {"norm": torch.full((1,), norm, dtype=dd), "grads": [torch.mul(g.to(dd), coef) for g in s["grads"]]}
