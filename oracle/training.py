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
