"""The training operators around the expert MLP, as they are measured: the
router's balance loss and its gradient, the backward pass of the router's
linear layer for dense logit gradients, and the orthogonalised momentum update
of the expert weights.

Each case is one pass through one operator.  `run` computes it in plain fp32
torch operations, or, where `own` is true, through the framework's entry
points.  Sizes are those of the framework's layers (tiny: 256 tokens, H = 128,
I = 256, 4 experts top-2; Mixtral: 16384 tokens, H = 4096, I = 14336, 8 experts
top-2; fine-grained: 8192 tokens, H = 2048, I = 1024, 64 experts top-8; up to
256 experts), and odd ones between them.
"""
import math

import torch

own = False

# the quintic of the Newton-Schulz iteration X <- a X + (b A + c A^2) X, A = X X^T
NS = (3.4445, -4.7750, 2.0315)
COEF = 0.01           # weight of the balance loss
MU = 0.95             # momentum of the update


def listed():
    return [
        # the smallest balance loss: a ragged handful of tokens (latency)
        {"name": "balance_fwd_77x5", "op": "balance_fwd", "T": 77, "E": 5, "k": 1, "mask": False, "disabled": 0},
        # the widest router on a long batch with padding tokens and experts switched off
        {"name": "balance_fwd_65536x256", "op": "balance_fwd", "T": 65536, "E": 256, "k": 8, "mask": True,
         "disabled": 3},
        # the fine-grained layer: gradient of the loss and of the route together
        {"name": "balance_bwd_8192x64", "op": "balance_bwd", "T": 8192, "E": 64, "k": 8, "mask": True, "disabled": 0,
         "route": True},
        # an odd expert count on an odd number of tokens, the loss's gradient alone
        {"name": "balance_bwd_30011x60", "op": "balance_bwd", "T": 30011, "E": 60, "k": 4, "mask": False,
         "disabled": 2, "route": False},
        # the tiny layer's router (latency)
        {"name": "router_bwd_256x128x4", "op": "router_bwd", "T": 256, "H": 128, "E": 4, "dx_in": True},
        # the Mixtral layer's router: the x and dx streams
        {"name": "router_bwd_16384x4096x8", "op": "router_bwd", "T": 16384, "H": 4096, "E": 8, "dx_in": True},
        # the fine-grained layer's router on an odd number of tokens, and the widest one
        {"name": "router_bwd_8191x2048x64", "op": "router_bwd", "T": 8191, "H": 2048, "E": 64, "dx_in": True},
        {"name": "router_bwd_5003x1024x256", "op": "router_bwd", "T": 5003, "H": 1024, "E": 256, "dx_in": False},
        # the update of the tiny layer's W_down (latency), an odd matrix that is taller than wide
        # with fp32 gradients, the fine-grained layer's W_down with the weights updated in the same call,
        # and one Mixtral expert's W_gate_up from its fp32 main_grad
        {"name": "muon_4x128x256", "op": "muon", "B": 4, "rows": 128, "cols": 256, "f32": False, "apply": False},
        {"name": "muon_3x1001x333", "op": "muon", "B": 3, "rows": 1001, "cols": 333, "f32": True, "apply": False},
        {"name": "muon_64x2048x1024", "op": "muon", "B": 64, "rows": 2048, "cols": 1024, "f32": False, "apply": True},
        {"name": "muon_1x28672x4096", "op": "muon", "B": 1, "rows": 28672, "cols": 4096, "f32": True, "apply": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance_fwd", "balance_bwd", "router_bwd", "muon", "muon"])
    if op in ("balance_fwd", "balance_bwd"):
        E = _log(rng, 2, 256)
        c = {"op": op, "T": _log(rng, 1, 65536), "E": E, "k": rng.randint(1, min(8, E)), "mask": rng.random() < 0.5}
        c["disabled"] = rng.randint(0, min(3, E - c["k"]))
        if op == "balance_bwd":
            c["route"] = rng.random() < 0.5
        return c
    if op == "router_bwd":
        return {"op": op, "T": _log(rng, 1, 16384), "H": 128 * _log(rng, 1, 32), "E": _log(rng, 2, 256),
                "dx_in": rng.random() < 0.5}
    top = _products(64, 2048, 1024)
    while True:
        c = {"op": op, "B": _log(rng, 1, 64), "rows": _log(rng, 8, 8192), "cols": _log(rng, 8, 8192),
             "f32": rng.random() < 0.5, "apply": rng.random() < 0.5}
        if _products(c["B"], c["rows"], c["cols"]) <= top and c["B"] * c["rows"] * c["cols"] <= 64 * 2048 * 1024:
            return c


def _products(B, rows, cols):
    """Multiply-adds x 2 of five steps: X X^T and A^2 are symmetric, so half of each is enough."""
    m, n = min(rows, cols), max(rows, cols)
    return 5.0 * B * (3.0 * m * m * n + float(m) ** 3)


def work(case):
    op = case["op"]
    if op == "balance_fwd":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 4 * T * k + (T if case["mask"] else 0) + 8 * E + 8, "flops": 6 * T * E}
    if op == "balance_bwd":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 8 * T * E + (T if case["mask"] else 0) + 4 * E + 4 + (12 * T * k if case["route"] else 0),
                "flops": 9 * T * E}
    if op == "router_bwd":
        T, H, E = case["T"], case["H"], case["E"]
        return {"bytes": 2 * T * H * (3 if case["dx_in"] else 2) + 4 * T * E + 6 * E * H, "flops": 4 * T * H * E}
    n = case["B"] * case["rows"] * case["cols"]
    # gradient and momentum read, momentum written, the update (or the weights, read and written) written
    return {"bytes": n * ((4 if case["f32"] else 2) + 8 + (4 if case["apply"] else 2)),
            "flops": _products(case["B"], case["rows"], case["cols"])}


# ------------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    op = case["op"]
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if op in ("balance_fwd", "balance_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        logits = normal(T, E, std=1.5) + normal(1, E)                  # some experts are preferred
        if case["disabled"]:
            logits[:, E - case["disabled"]:] = float("-inf")
        s["logits"] = logits.contiguous()
        top = torch.topk(logits, k, dim=1)
        s["ids"] = top.indices.to(torch.int32).contiguous()
        s["mask"] = None
        if case["mask"]:                                               # the padding of a batch: about an eighth
            s["mask"] = torch.rand(T, generator=g, device="cuda") >= 0.125
        if op == "balance_bwd":
            keep = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
            s["counts"] = torch.bincount(s["ids"][keep].reshape(-1).long(), minlength=E).to(torch.int32)
            s["n_tokens"] = keep.sum().to(torch.int32).reshape(1)
            s["dloss"] = torch.full((1,), 0.5, device="cuda")
            s["dlogits"] = torch.empty((T, E), device="cuda")
            s["probs"] = s["dprobs"] = None
            if case["route"]:
                e = torch.exp(top.values - top.values[:, :1])
                s["probs"] = (e / e.sum(1, keepdim=True)).contiguous()
                # of the size of the loss's own gradient, so that both show in the sum
                s["dprobs"] = normal(T, k, std=0.01 / max(T, 1))
        else:
            s["loss"] = torch.empty(1, device="cuda")
            s["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
            s["prob_sums"] = torch.empty(E, device="cuda")
            s["n_tokens"] = torch.empty(1, dtype=torch.int32, device="cuda")
        return s
    if op == "router_bwd":
        T, H, E = case["T"], case["H"], case["E"]
        s["x"] = normal(T, H).bfloat16()
        s["w"] = normal(E, H, std=0.02).bfloat16()
        d = normal(T, E, std=1e-3)                                     # the loss's dense part ...
        d += normal(T, E, std=2e-2) * (torch.rand(T, E, generator=g, device="cuda") < 2.0 / E)   # ... and chosen experts
        s["dlogits"] = d
        s["dx_in"] = normal(T, H, std=1e-3).bfloat16() if case["dx_in"] else None
        s["dx"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        s["dw"] = torch.empty((E, H), device="cuda")
        return s
    B, m, n = case["B"], case["rows"], case["cols"]
    r = max(1, min(m, n) // 16)

    def gradient():                                                    # a few strong directions over noise
        u = normal(B, m, r) @ (normal(B, r, n) * (2.0 / math.sqrt(r)))
        return (u + normal(B, m, n)) * 1e-3

    grad = gradient()
    momentum = gradient() * 4.0 + grad * 6.0
    if B > 2:                                                          # an expert that got no token yet
        grad[1] = 0.0
        momentum[1] = 0.0
    s["grad"] = grad.contiguous() if case["f32"] else grad.bfloat16()
    s["momentum"] = momentum.contiguous()
    s["momentum_out"] = torch.empty_like(momentum)
    s["out"] = torch.empty((B, m, n), dtype=torch.bfloat16, device="cuda")
    s["weights"] = normal(B, m, n, std=0.02).bfloat16() if case["apply"] else None
    s["scale"] = 0.2 * math.sqrt(max(m, n))
    # a rate at which the update shows beside the weights
    s["lr"], s["decay"] = 0.05, 0.1
    return s


# --------------------------------------------------------------- plain forms --

def _softmax(logits):
    top = logits.max(dim=1, keepdim=True).values
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = torch.exp(logits - top)
    total = e.sum(dim=1, keepdim=True)
    return torch.where(total > 0, e / total, torch.zeros_like(e))


def _plain_balance_fwd(s):
    T, E, k = s["case"]["T"], s["case"]["E"], s["case"]["k"]
    p = _softmax(s["logits"])
    if s["mask"] is None:
        hits = s["ids"].reshape(-1).long()
        one = torch.ones_like(hits)
        n = torch.full((1,), T, dtype=torch.int32, device=p.device)
    else:
        p = p * s["mask"][:, None]
        hits = s["ids"].reshape(-1).long()
        one = s["mask"][:, None].expand(T, k).reshape(-1).long()
        n = s["mask"].sum().to(torch.int32).reshape(1)
    counts = torch.zeros(E, dtype=torch.int64, device=p.device).index_add_(0, hits, one)
    prob_sums = p.sum(dim=0)
    nf = n.float().clamp(min=1.0)
    loss = (COEF * E) * ((counts.float() / (k * nf)) * (prob_sums / nf)).sum().reshape(1)
    return {"loss": loss, "counts": counts.to(torch.int32), "prob_sums": prob_sums, "n_tokens": n}


def _plain_balance_bwd(s):
    E, k = s["case"]["E"], s["case"]["k"]
    p = _softmax(s["logits"])
    nf = s["n_tokens"].float().clamp(min=1.0)
    f = s["counts"].float() / (k * nf)
    d = (s["dloss"] * COEF * E / nf) * p * (f - (p * f).sum(dim=1, keepdim=True))
    if s["mask"] is not None:
        d = d * s["mask"][:, None]
    if s["probs"] is not None:
        q = s["probs"]
        dq = q * (s["dprobs"] - (q * s["dprobs"]).sum(dim=1, keepdim=True))
        d = d.scatter_add(1, s["ids"].long(), dq)
    return d


def _plain_router_bwd(s):
    d = s["dlogits"]
    dx = d @ s["w"].float()
    if s["dx_in"] is not None:
        dx = dx + s["dx_in"].float()
    return {"dx": dx.bfloat16(), "dw": d.t() @ s["x"].float()}


def _ns_step(x):
    gram = x @ x.transpose(1, 2)
    return NS[0] * x + (NS[1] * gram + NS[2] * (gram @ gram)) @ x


def _plain_muon(s):
    g = s["grad"].float()
    mom = MU * s["momentum"] + g
    u = g + MU * mom
    tall = u.shape[1] > u.shape[2]
    if tall:
        u = u.transpose(1, 2)
    norm = torch.sqrt((u * u).sum(dim=(1, 2), keepdim=True))
    x = torch.where(norm > 0, u / norm, torch.zeros_like(u))
    x = _ns_step(_ns_step(_ns_step(_ns_step(_ns_step(x)))))
    if tall:
        x = x.transpose(1, 2)
    x = x * s["scale"]
    if s["weights"] is not None:
        x = s["weights"].float() * (1.0 - s["lr"] * s["decay"]) - s["lr"] * x
    return {"out": x.contiguous().bfloat16(), "momentum": mom}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"balance_fwd": _plain_balance_fwd, "balance_bwd": _plain_balance_bwd, "router_bwd": _plain_router_bwd,
                "muon": _plain_muon}[op](s)
    import mxfp8_grouped_gemm_gb300 as mxg
    if op == "balance_fwd":
        mxg.mxg_balance_loss_fwd(s["logits"], s["ids"], COEF, s["status"], token_mask=s["mask"], loss=s["loss"],
                                 counts=s["counts"], prob_sums=s["prob_sums"], n_tokens=s["n_tokens"])
        return {"loss": s["loss"], "counts": s["counts"], "prob_sums": s["prob_sums"], "n_tokens": s["n_tokens"]}
    if op == "balance_bwd":
        route = (s["ids"], s["probs"], s["dprobs"]) if s["probs"] is not None else None
        return mxg.mxg_balance_loss_bwd(s["logits"], s["counts"], s["n_tokens"], c["k"], COEF, s["status"],
                                        dloss=s["dloss"], token_mask=s["mask"], route=route, dlogits=s["dlogits"])
    if op == "router_bwd":
        mxg.mxg_router_linear_bwd(s["x"], s["w"], s["dlogits"], s["dx_in"], s["status"], dx=s["dx"],
                                  dw_router=s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if c["apply"]:
        mxg.mxg_muon_update(s["grad"], s["status"], momentum=s["momentum"], momentum_out=s["momentum_out"], mu=MU,
                            nesterov=True, steps=5, coefficients=NS, scale=s["scale"], weights=s["weights"],
                            weights_out=s["out"], lr=s["lr"], weight_decay=s["decay"])
    else:
        mxg.mxg_muon_update(s["grad"], s["status"], momentum=s["momentum"], momentum_out=s["momentum_out"], mu=MU,
                            nesterov=True, steps=5, coefficients=NS, scale=s["scale"], update=s["out"])
    return {"out": s["out"], "momentum": s["momentum_out"]}


# ------------------------------------------------------------------ 64 bits --

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("balance_fwd", "balance_bwd"):
        E, k = case["E"], case["k"]
        z = s["logits"].double()
        w = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))         # every row keeps at least k finite logits
        live = torch.ones_like(z[:, 0]) if s["mask"] is None else s["mask"].double()
        n = float(live.sum())
        if op == "balance_fwd":
            sums = torch.einsum("te,t->e", w, live)
            share = torch.einsum("tke,t->e", torch.nn.functional.one_hot(s["ids"].long(), E).double(), live)
            loss = COEF * E * torch.dot(share, sums) / (k * n * n) if n else torch.zeros((), device="cuda").double()
            return {"loss": loss.reshape(1), "counts": None, "prob_sums": sums, "n_tokens": None}
        f = s["counts"].double() / (k * max(n, 1.0))
        centred = f[None, :] - torch.einsum("te,e->t", w, f)[:, None]
        d = w * centred * live[:, None] * (float(s["dloss"]) * COEF * E / max(n, 1.0))
        if s["probs"] is not None:
            q, dq = s["probs"].double(), s["dprobs"].double()
            part = q * dq - q * torch.einsum("tk,tk->t", q, dq)[:, None]
            d = d + torch.einsum("tk,tke->te", part, torch.nn.functional.one_hot(s["ids"].long(), E).double())
        return d
    if op == "router_bwd":
        d = s["dlogits"].double()
        dx = torch.einsum("te,eh->th", d, s["w"].double())
        if s["dx_in"] is not None:
            dx += s["dx_in"].double()
        return {"dx": dx, "dw": torch.einsum("te,th->eh", d, s["x"].double())}
    m, n = min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    if 5.0 * case["B"] * (4.0 * m * m * n + 2.0 * float(m) ** 3) > 4e12:
        return None
    mom = s["momentum"].double() * MU + s["grad"].double()
    y = s["grad"].double() + MU * mom
    if case["rows"] < case["cols"]:
        y = y.transpose(1, 2)
    size = y.flatten(1).norm(dim=1)
    y = y / torch.where(size > 0, size, torch.ones_like(size))[:, None, None]
    a, b, c = NS
    eye = torch.eye(m, dtype=torch.float64, device="cuda")
    for _ in range(5):                                                 # tall form: Y <- Y (a + b S + c S^2), S = Y^T Y
        small = torch.bmm(y.transpose(1, 2), y)
        y = torch.bmm(y, a * eye + torch.bmm(small, b * eye + c * small))
    if case["rows"] < case["cols"]:
        y = y.transpose(1, 2)
    y = y * s["scale"]
    if s["weights"] is not None:
        y = s["weights"].double() * (1.0 - s["lr"] * s["decay"]) - s["lr"] * y
    return {"out": y.contiguous(), "momentum": mom}
