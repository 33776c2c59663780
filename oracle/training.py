"""fp64 oracle of the training operators around the expert MLP: the router's
balance loss and its gradient, the router linear layer's backward for dense
logit gradients, and the orthogonalised momentum update.  Written from the
formulas in numpy, sharing no code with the GPU path."""
import numpy as np


def softmax_rows(logits):
    """Softmax over each row; a row without a finite logit is all zeros."""
    z = np.asarray(logits, dtype=np.float64)
    top = z.max(axis=1, keepdims=True)
    top = np.where(np.isneginf(top), 0.0, top)
    with np.errstate(invalid="ignore"):
        e = np.exp(z - top)
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=~(s == 0.0))


def balance_loss(logits, ids, coef, mask=None):
    """-> (loss, counts [E], prob_sums [E], n)."""
    T, E = logits.shape
    k = ids.shape[1]
    live = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    n = int(live.sum())
    p = softmax_rows(np.where(live[:, None], logits, -np.inf))
    chosen = ids[live].reshape(-1)
    chosen = chosen[(chosen >= 0) & (chosen < E)]
    counts = np.bincount(chosen, minlength=E)
    sums = p.sum(axis=0)
    loss = coef * E * float(np.dot(counts / (k * n), sums / n)) if n else 0.0
    return loss, counts, sums, n


def route_grad(ids, probs, dprobs, E):
    """Gradient of the chosen logits through the softmax over them, dense [T, E]."""
    q, dq = np.asarray(probs, np.float64), np.asarray(dprobs, np.float64)
    d = q * (dq - (q * dq).sum(axis=1, keepdims=True))
    out = np.zeros((ids.shape[0], E))
    t, j = np.nonzero((ids >= 0) & (ids < E))
    np.add.at(out, (t, ids[t, j]), d[t, j])
    return out


def balance_grad(logits, counts, n, k, coef, dloss=1.0, mask=None):
    """d loss / d logits with the counts held fixed, [T, E]."""
    T, E = logits.shape
    if n == 0:
        return np.zeros((T, E))
    live = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    p = softmax_rows(np.where(live[:, None], logits, -np.inf))
    f = np.asarray(counts, np.float64) / (float(k) * n)
    return dloss * coef * E / n * p * (f[None, :] - (p @ f)[:, None])


def router_linear_bwd(x, w, g, dx_in=None):
    """Logits = x w^T with logit gradients g -> (dx, dw)."""
    dx = g @ w
    return (dx if dx_in is None else dx + dx_in), g.T @ x


def momentum(grad, mom, mu, nesterov):
    """-> (new momentum, u)."""
    new = mu * mom + grad
    return new, (grad + mu * new if nesterov else new)


def orthogonalise(u, steps, coefficients):
    """Newton-Schulz iterations on one matrix."""
    a, b, c = coefficients
    norm = np.sqrt((u * u).sum())
    if norm == 0.0:
        return np.zeros_like(u)
    x = u / norm
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.T if tall else x


def _fp16_parts(v, scale, parts):
    """v as the sum of one or two fp16 numbers held times `scale`."""
    out, rest = [], np.asarray(v, np.float64) * scale
    for _ in range(parts):
        h = rest.astype(np.float16).astype(np.float64)
        out.append(h / scale)
        rest = rest - h
    return out


def bf16_round(v):
    """Nearest bf16 value (ties to even) of each finite element."""
    u = np.ascontiguousarray(v, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)


def orthogonalise_in_fp16(u, steps, coefficients, x_parts, b_parts, lost=None):
    """`orthogonalise` in the GPU's number format, all else in 64 bits: X and A in x_parts fp16 numbers, B in b_parts
    (X times the power of two next to sqrt(long side), A and B times 2^12), low parts multiplied by high ones only,
    the result rounded to bf16.  It tells what of an update's error is the format's own.  lost = (product, i, j) leaves
    out part i of its first operand times part j of its second, for tests of what a bound can see."""
    a, b, c = coefficients
    x = u / np.sqrt((u * u).sum())
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    sx = 1
    while sx * sx < x.shape[1]:
        sx *= 2

    def product(name, p, q):
        return sum(p[i] @ q[j] for i in range(len(p)) for j in range(len(q)) if i + j < 2 and (name, i, j) != lost)

    xp = _fp16_parts(x, sx, x_parts)
    for _ in range(steps):
        ap = _fp16_parts(product("A", xp, [v.T for v in xp]), 4096.0, x_parts)
        bp = _fp16_parts(a * np.eye(x.shape[0]) + b * sum(ap) + c * product("B", ap, ap), 4096.0, b_parts)
        x = product("X", bp, xp)
        xp = _fp16_parts(x, sx, x_parts)
    return bf16_round(x.T if tall else x)
