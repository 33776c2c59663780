"""fp64 oracle of the operators around the expert MLP in a block of a model:
the residual norm and its backward, routing by scores and its gradient, the
norm over all gradients.  Written from the formulas in numpy, sharing no code
with the GPU path."""
import numpy as np


def rms_norm(x, weight, eps, residual=None):
    """-> (r, rstd [T], y), nothing rounded."""
    r = np.asarray(x, np.float64) if residual is None else np.asarray(x, np.float64) + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(r * r, axis=1) + eps)
    return r, rstd, r * rstd[:, None] * np.asarray(weight, np.float64)


def rms_norm_grad(dy, r, weight, rstd, dresidual=None):
    """-> (gradient of r, gradient of weight)."""
    dy, r, rstd = (np.asarray(a, np.float64) for a in (dy, r, rstd))
    xh = r * rstd[:, None]
    g = dy * np.asarray(weight, np.float64)
    d = rstd[:, None] * (g - xh * np.mean(g * xh, axis=1, keepdims=True))
    return (d if dresidual is None else d + np.asarray(dresidual, np.float64)), (dy * xh).sum(axis=0)


def scores(logits, kind):
    z = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z))
        top = z.max(axis=1, keepdims=True)
        e = np.exp(z - np.where(np.isneginf(top), 0.0, top))
        s = e.sum(axis=1, keepdims=True)
        return np.divide(e, s, out=np.zeros_like(e), where=~(s == 0.0))


def _order(values):
    """Indices from the largest value to the smallest, equal ones by index."""
    return np.argsort(-values, axis=1, kind="stable")


def route(logits, k, kind, bias=None, groups=1, top_groups=1, group_top=2, renormalize=True, scale=1.0):
    """-> (ids [T, k], weights [T, k])."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    s = scores(z, kind)
    by_score = bias is not None or (top_groups < groups and group_top == 2)
    with np.errstate(invalid="ignore"):
        c = z if not by_score else s if bias is None else s + np.asarray(bias, np.float64)
    c = np.where(np.isneginf(z) | np.isnan(c), -np.inf, c)
    kept = np.ones((T, E), bool)
    if top_groups < groups:
        size = E // groups
        best = -np.sort(-c.reshape(T, groups, size), axis=2)[:, :, :group_top]
        live = ~np.isneginf(best)
        value = np.where(live.any(axis=2), np.where(live, best, 0.0).sum(axis=2), -np.inf)
        chosen = _order(value)[:, :top_groups]
        kept = np.zeros((T, groups), bool)
        np.put_along_axis(kept, chosen, True, axis=1)
        kept = np.repeat(kept, size, axis=1)
    # the kept experts first, in order of c, equal ones by id
    ids = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -c, ~kept), axis=1)[:, :k]
    w = np.take_along_axis(s, ids, axis=1)
    if renormalize:
        if kind == "softmax":                        # over the chosen logits: the same, where all scores vanish too
            w = scores(np.take_along_axis(z, ids, axis=1), "softmax")
        else:                                        # through log sigmoid(z), which holds scores far below 1e-308
            v = np.take_along_axis(z, ids, axis=1)
            w = scores(np.minimum(v, 0.0) - np.log1p(np.exp(-np.abs(v))), "softmax")
    return ids, w * scale


def route_grad(logits, ids, probs, dprobs, kind, renormalize=True, scale=1.0, add=None):
    """Gradient of the weights on the logits, [T, E]; ids out of range add nothing at an expert."""
    z, p, dp = (np.asarray(a, np.float64) for a in (logits, probs, dprobs))
    T, E = z.shape
    s = scores(z, kind)
    S = (p * dp).sum(axis=1, keepdims=True)
    d = p * (dp - S / scale) if renormalize else p * dp
    out = np.zeros((T, E)) if add is None else np.array(add, np.float64)
    t, j = np.nonzero((ids >= 0) & (ids < E))
    e = ids[t, j]
    np.add.at(out, (t, e), d[t, j] * (1.0 / (1.0 + np.exp(z[t, e])) if kind == "sigmoid" else 1.0))
    if kind == "softmax" and not renormalize:
        out -= s * S
    return out


def grad_norm(grads):
    """Square root of the sum of all squares, safe for any finite fp32 values."""
    top = max((float(np.abs(g).max(initial=0.0)) for g in grads), default=0.0)
    if top == 0.0 or not np.isfinite(top):
        return top
    return top * np.sqrt(sum(float(((np.asarray(g, np.float64) / top) ** 2).sum()) for g in grads))
