"""Routing by scores and its gradient on the GPU against the fp64 oracle: ids
equal, weights and gradients within bounds on the fp32 arithmetic."""
import numpy as np
import pytest
import torch

from gpu_helpers import np_, require_gpu
from oracle import block

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CASES = [   # T, E, k, kind, bias, groups, top_groups, group_top, renormalize, scale
    (1, 1, 1, "softmax", None, 1, 1, 1, True, 1.0),
    (1, 2, 2, "sigmoid", 0.1, 1, 1, 1, False, 1.0),
    (77, 5, 1, "softmax", 0.1, 1, 1, 1, False, 2.5),
    (300, 8, 2, "softmax", None, 1, 1, 1, True, 1.0),
    (65, 8, 8, "sigmoid", 0.2, 4, 4, 2, True, 1.0),          # every expert chosen
    (1001, 9, 3, "sigmoid", 0.1, 3, 2, 2, True, 2.5),        # one past a lane, groups across lanes
    (999, 17, 4, "softmax", 0.01, 17, 9, 1, True, 1.0),      # groups of one
    (640, 30, 6, "sigmoid", None, 5, 2, 2, False, 1.0),      # sums over groups without a bias
    (640, 30, 6, "softmax", None, 5, 2, 1, False, 1.5),      # the groups' largest without a bias
    (2000, 60, 4, "sigmoid", 0.05, 10, 3, 2, True, 1.0),
    (4096, 64, 8, "softmax", None, 1, 1, 1, False, 1.0),
    (2048, 64, 8, "softmax", 0.02, 8, 3, 2, True, 1.0),
    (515, 100, 32, "sigmoid", 0.3, 4, 2, 1, True, 1.0),
    (700, 128, 16, "sigmoid", 0.1, 64, 32, 2, False, 2.0),   # groups of two
    (130, 129, 8, "softmax", 0.001, 3, 2, 2, True, 1.0),
    (5000, 256, 8, "sigmoid", 0.05, 8, 4, 2, True, 2.5),     # the widest
    (300, 256, 32, "softmax", 0.001, 16, 8, 1, False, 1.0),
    (300, 256, 8, "sigmoid", 0.05, 256, 100, 1, True, 1.0),
]
IDS = [f"{c[0]}x{c[1]}k{c[2]}{c[3]}" + ("" if c[4] is None else "b") + f"g{c[5]}" for c in CASES]


def _inputs(T, E, k, bias, seed=0, std=2.0):
    rng = np.random.default_rng(1000 * E + T + seed)
    z = (rng.standard_normal((T, E)) * std + rng.standard_normal((1, E))).astype(np.float32)
    b = None if bias is None else (rng.standard_normal(E) * bias).astype(np.float32)
    return z, b, rng


def _dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _options(case):
    _, _, k, kind, _, groups, top_groups, group_top, renormalize, scale = case
    return dict(score=kind, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renormalize,
                scale=scale)


def _rel(z, k, kind, renormalize):
    """Relative error of a weight.  exp is within 2 ulp (4 U) of an argument that rounds once (spread * U); a sigmoid adds
    an addition and a quotient (2).  Sums of up to 256 scores are 8 in a row and 5 halvings, of the k chosen 8 and 5;
    quotient, factor and its product 3, the scaled sigmoid's second exponential 4."""
    finite = z[np.isfinite(z)]
    spread = float(finite.max() - finite.min()) if finite.size else 0.0
    return ((spread if kind == "softmax" or renormalize else 0.0) + 2 * (4 + 2) + 13 + 13 + 3 + 4) * U


def _check(m, z, b, k, opts):
    ids, probs = m.mxg_route_scores_fwd(_dev(z), k, bias=_dev(b), **opts)
    torch.cuda.synchronize()
    kind = opts.get("score", "softmax")
    ref, w = block.route(z, k, kind, b, opts.get("groups", 1), opts.get("top_groups", 1), opts.get("group_top", 2),
                         opts.get("renormalize", True), opts.get("scale", 1.0))
    assert np.array_equal(np_(ids), ref)
    assert (np.abs(np_(probs) - w) <= _rel(z, k, kind, opts.get("renormalize", True)) * w + 1e-37).all()
    return ref, w


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_route_fwd(case):
    m = require_gpu()
    T, E, k, kind, bias = case[:5]
    z, b, _ = _inputs(T, E, k, bias)
    _check(m, z, b, k, _options(case))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_route_fwd_with_experts_off(case):
    """Masked logits: single experts, whole groups, all but fewer than k, whole rows; biases of -inf."""
    m = require_gpu()
    T, E, k, kind, bias = case[:5]
    z, b, rng = _inputs(T, E, k, bias, seed=1)
    z[rng.random((T, E)) < 0.3] = -np.inf
    z[::7] = -np.inf
    if T > 2:
        z[2, 1:] = -np.inf
    z[T // 2:, 0] = -np.finfo(np.float32).max            # a mask of the type's lowest value ranks before -inf
    if b is not None and E > k:
        b[E // 2] = -np.inf
    _check(m, z, b, k, _options(case))


@pytest.mark.parametrize("case", [c for c in CASES if c[1] > 4], ids=[i for i, c in zip(IDS, CASES) if c[1] > 4])
def test_route_fwd_between_neighbouring_numbers(case):
    """Ids where fp32 scores cannot decide: logits an ulp or nothing apart, biases of the size of the steps."""
    m = require_gpu()
    T, E, k, kind, bias = case[:5]
    rng = np.random.default_rng(E + T)
    z = (0.25 + rng.integers(0, 4, (T, E)) * np.float32(2.0 ** -24)).astype(np.float32)
    b = None if bias is None else (rng.integers(0, 3, E) * np.float32(2.0 ** -25)).astype(np.float32)
    _check(m, z, b, k, _options(case))
    z = rng.integers(-1, 2, (T, E)).astype(np.float32) * np.float32(0.5)          # equal ones, and -0 beside 0
    z[rng.random((T, E)) < 0.5] *= -1.0
    _check(m, z, b, k, _options(case))
    _check(m, np.zeros((T, E), np.float32), b, k, _options(case))                # padding


@pytest.mark.parametrize("E,groups,top_groups,k", [(8, 4, 2, 4), (30, 10, 4, 9), (96, 32, 10, 20), (255, 85, 30, 32)])
def test_route_fwd_equal_logits_in_and_out_of_the_groups(E, groups, top_groups, k):
    """Small groups of a lane with distinct maxima: what they hold besides is equal, kept or not."""
    m = require_gpu()
    rng = np.random.default_rng(E)
    T, size = 200, E // groups
    z = np.ones((T, groups, size), np.float32)
    z[rng.random(z.shape) < 0.3] = 0.5
    z[:, :, size - 1] = 2.0 + rng.permuted(np.tile(np.arange(groups), (T, 1)), axis=1)
    for bias in (None, np.zeros(E, np.float32)):
        _check(m, z.reshape(T, E), bias, k, dict(groups=groups, top_groups=top_groups, group_top=1))


@pytest.mark.parametrize("E,groups,top_groups,k", [(16, 2, 1, 4), (32, 2, 1, 5), (64, 8, 3, 14), (256, 8, 2, 32)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_fwd_groups_with_few_experts_left(E, groups, top_groups, k, group_top):
    """Most experts off: what fills the route comes from the groups that take part, never from the others."""
    m = require_gpu()
    rng = np.random.default_rng(E + group_top)
    z = rng.standard_normal((500, E)).astype(np.float32)
    z[rng.random(z.shape) < 0.8] = -np.inf
    bias = (rng.standard_normal(E) * 0.3).astype(np.float32)
    for kind in ("softmax", "sigmoid"):
        for b in (None, bias):
            _check(m, z, b, k, dict(score=kind, groups=groups, top_groups=top_groups, group_top=group_top))


@pytest.mark.parametrize("E,groups,top_groups,k", [(8, 1, 1, 3), (16, 2, 1, 8), (64, 8, 2, 9), (30, 5, 2, 12), (256, 8, 4, 8)])
def test_route_fwd_infinite_biases(E, groups, top_groups, k):
    """Experts that are always chosen (a bias of +inf), in one group and in several, beside some that never are."""
    m = require_gpu()
    rng = np.random.default_rng(E)
    z = rng.standard_normal((300, E)).astype(np.float32)
    z[rng.random(z.shape) < 0.1] = -np.inf
    for always in (1, 2, E // 2, E):
        bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
        bias[rng.choice(E, always, replace=False)] = np.inf
        if always < E:
            bias[rng.choice(np.flatnonzero(np.isfinite(bias)))] = -np.inf
        for group_top in (1, 2):
            if group_top <= E // groups:
                _check(m, z, bias, k, dict(score="sigmoid", groups=groups, top_groups=top_groups, group_top=group_top))


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [30.0, 60.0, 1e4])
def test_route_fwd_far_logits(kind, size):
    """Scores next to 0 and 1, and beyond what fp32 holds."""
    m = require_gpu()
    rng = np.random.default_rng(7)
    z = (rng.standard_normal((400, 32)) * size).astype(np.float32)
    z[100:200] = -np.abs(z[100:200]) - size
    z[200:300] = np.abs(z[200:300]) + size
    b = (rng.standard_normal(32) * 0.1).astype(np.float32)
    for bias, opts in ((None, {}), (b, {}), (b, {"groups": 4, "top_groups": 2}), (1e4 * b, {}), (b, {"renormalize": False})):
        ids, probs = m.mxg_route_scores_fwd(_dev(z), 4, score=kind, bias=_dev(bias), **opts)
        ref, w = block.route(z, 4, kind, bias, opts.get("groups", 1), opts.get("top_groups", 1), 2,
                             opts.get("renormalize", True))
        assert np.array_equal(np_(ids), ref)
        ok = np.isfinite(np_(probs)).all()
        assert ok
        if kind == "softmax" or size < 100:              # oracle's own e^z leaves fp64 beyond
            rel = (4 * size * 2 + 60) * U
            keep = w > 1e-30
            assert (np.abs(np_(probs) - w)[keep] <= (rel * w)[keep]).all()


def test_route_fwd_nan_and_infinity():
    m = require_gpu()
    z = np.tile(np.arange(8, dtype=np.float32), (4, 1))
    z[0, 7] = np.nan
    z[1, 2] = np.inf
    z[2] = np.nan
    for kind in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(8, device="cuda")):
            ids, probs = m.mxg_route_scores_fwd(_dev(z), 3, score=kind, bias=bias)
            ids, probs = np_(ids), np_(probs)
            assert ((ids >= 0) & (ids < 8)).all() and all(len(set(r)) == 3 for r in ids.tolist())
            assert ids[2].tolist() == [0, 1, 2] and np.isnan(probs[2]).all()
            assert ids[3].tolist() == [7, 6, 5]
            if bias is None or kind == "sigmoid":
                assert ids[0].tolist() == [6, 5, 4] and np.isfinite(probs[0]).all()
                assert ids[1].tolist() == [2, 7, 6]


def test_route_fwd_is_the_plain_route():
    """Softmax, renormalised, without bias or groups is mxg_route_topk."""
    m = require_gpu()
    z = _inputs(3000, 64, 8, None)[0]
    ids, probs = m.mxg_route_scores_fwd(_dev(z), 8)
    ids2, probs2 = m.mxg_route_topk(_dev(z), 8)
    assert torch.equal(ids, ids2)
    assert float((probs - probs2).abs().max()) <= 40 * U


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_route_bwd(case, add):
    m = require_gpu()
    T, E, k, kind, bias, groups, top_groups, group_top, renormalize, scale = case
    z, b, rng = _inputs(T, E, k, bias, seed=2)
    z[rng.random((T, E)) < 0.1] = -np.inf
    ids, p = block.route(z, k, kind, b, groups, top_groups, group_top, renormalize, scale)
    p = p.astype(np.float32)
    dp = (rng.standard_normal((T, k)) * 0.01).astype(np.float32)
    base = (rng.standard_normal((T, E)) * 1e-3).astype(np.float32) if add else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    into = _dev(base)
    got = m.mxg_route_scores_bwd(_dev(z), _dev(ids.astype(np.int32)), _dev(p), _dev(dp), st, score=kind,
                                 renormalize=renormalize, scale=scale, dlogits_in=into, dlogits=into)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and (into is None or got is into)
    # the oracle takes S over the weights as they are given; renormalised ones sum to scale within their rounding
    ref = block.route_grad(z, ids, p, dp, kind, renormalize, scale, base)
    S = (np.abs(p * dp).astype(np.float64)).sum(axis=1, keepdims=True)
    far = 2 * np.abs(dp).max(axis=1, keepdims=True).astype(np.float64)       # |dp_j - dp_0|
    # a difference (1), a sum of up to 8 + 5 products, times 1 / scale (2), a difference, the product; the sum of the
    # weights is off by k / 2 + 1 roundings where it should be scale; a sigmoid is within 6
    at = np.abs(p) * (np.abs(dp) + far + S / scale) * (3 + 14 + 3 + k / 2 + 1 + 3 + 6) * U
    bound = np.zeros((T, E))
    np.put_along_axis(bound, ids, at, axis=1)
    if kind == "softmax" and not renormalize:
        spread = float(z[np.isfinite(z)].max() - z[np.isfinite(z)].min())
        bound += block.scores(z, kind) * S * (spread + 4 + 13 + 14 + 4) * U
    assert (np.abs(np_(got) - ref) <= bound + 3 * U * (np.abs(ref) + (0 if base is None else np.abs(base))) + 1e-37).all()


def test_route_bwd_bad_and_double_ids():
    m = require_gpu()
    T, E = 40, 12
    z, _, rng = _inputs(T, E, 3, None)
    ids = rng.integers(0, E, (T, 3)).astype(np.int32)
    ids[::4, 1] = ids[::4, 0]
    p, dp = rng.random((T, 3)).astype(np.float32), rng.standard_normal((T, 3)).astype(np.float32)
    for kind in ("softmax", "sigmoid"):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = m.mxg_route_scores_bwd(_dev(z), _dev(ids), _dev(p), _dev(dp), st, score=kind, renormalize=False)
        ref = block.route_grad(z, ids, p, dp, kind, False)
        assert np.abs(np_(got) - ref).max() <= 100 * U * np.abs(ref).max() and int(st.item()) == 0
        for bad in (-1, E, 1 << 30):
            wrong = ids.copy()
            wrong[5, 2] = bad
            st.zero_()
            got = m.mxg_route_scores_bwd(_dev(z), _dev(wrong), _dev(p), _dev(dp), st, score=kind, renormalize=False)
            ref = block.route_grad(z, wrong, p, dp, kind, False)
            assert np.abs(np_(got) - ref).max() <= 100 * U * np.abs(ref).max()
            assert m.status_string(int(st.item())) == m.status_string(16)


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_gradient_is_the_difference(kind, renormalize):
    """The GPU gradient against central differences of the GPU's own choice in fp64."""
    m = require_gpu()
    T, E, k = 6, 20, 4
    z, b, rng = _inputs(T, E, k, 0.1)
    dp = rng.standard_normal((T, k)).astype(np.float32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, p = m.mxg_route_scores_fwd(_dev(z), k, score=kind, bias=_dev(b), renormalize=renormalize, scale=1.5)
    got = np_(m.mxg_route_scores_bwd(_dev(z), ids, p, _dev(dp), st, score=kind, renormalize=renormalize, scale=1.5))
    chosen = np_(ids).astype(np.int64)

    def loss(z):
        w = np.take_along_axis(block.scores(z, kind), chosen, axis=1)
        return (1.5 * (w / w.sum(axis=1, keepdims=True) if renormalize else w) * dp).sum()

    h = 1e-5
    for t in range(T):
        for e in range(0, E, 3):
            d = np.zeros((T, E))
            d[t, e] = h
            diff = (loss(z.astype(np.float64) + d) - loss(z.astype(np.float64) - d)) / (2 * h)
            assert abs(diff - got[t, e]) <= 1e-5


@pytest.mark.parametrize("E", [7, 64, 256])
def test_route_rows_behind_the_last_stay(E):
    m = require_gpu()
    T, k = 13, 3
    z = _dev(_inputs(T, E, k, None)[0])
    ids = torch.full((T + 4, k), 77, dtype=torch.int32, device="cuda")
    probs, d = torch.full((T + 4, k), 77.0, device="cuda"), torch.full((T + 4, E), 77.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.mxg_route_scores_fwd(z, k, score="sigmoid", bias=torch.zeros(E, device="cuda"), ids=ids[:T], probs=probs[:T])
    m.mxg_route_scores_bwd(z, ids[:T], probs[:T], probs[:T], st, score="sigmoid", dlogits=d[:T])
    assert bool((ids[T:] == 77).all()) and bool((probs[T:] == 77).all()) and bool((d[T:] == 77).all())


MASKS = [(-10.0, 1), (-1e4, 1), (-1e9, 1), (-1e9, 40), (1e4, 1), (1e4, 3), (-float(np.finfo(np.float32).max), 5)]


@pytest.mark.parametrize("E,groups,top_groups,group_top,k", [
    (256, 1, 1, 1, 8), (256, 8, 4, 2, 8), (256, 8, 4, 1, 8), (256, 128, 60, 2, 8), (64, 1, 1, 1, 8), (64, 8, 3, 2, 4),
    (64, 16, 6, 2, 8), (90, 9, 4, 2, 8), (90, 45, 20, 2, 5)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_fwd_large_finite_biases(kind, E, groups, top_groups, group_top, k):
    """A finite bias that keeps experts out or forces them in, beside small ones; in a group with one of the other sign
    the sum of the two is small, but not its error."""
    m = require_gpu()
    rng = np.random.default_rng(E + groups)
    z = (rng.standard_normal((700, E)) * 1.5).astype(np.float32)
    opts = dict(score=kind, groups=groups, top_groups=top_groups, group_top=group_top)
    for value, experts in MASKS:
        b = (rng.standard_normal(E) * 0.05).astype(np.float32)
        at = rng.choice(E, min(experts, E // 4), replace=False)
        b[at] = value
        _check(m, z, b, k, opts)
        if groups > 1:
            b[:] = (rng.standard_normal(E) * 0.05).astype(np.float32)
            size = E // groups
            for g in rng.choice(groups, max(groups // 2, 1), replace=False):           # |value| and -|value| in a group
                b[g * size:(g + 1) * size] = -abs(value)
                b[g * size] = abs(value)
            _check(m, z, b, k, opts)


def _time(call, n=20):
    """Shortest of n calls in us, on the GPU's clock."""
    best = float("inf")
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 4), (16, 8)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_fwd_a_masked_expert_costs_nothing(kind, groups, top_groups):
    """Experts far from every decision do not send the others' to 64 bits: the same call with one bias of -1e9 (or +1e4,
    or +inf) takes at most half as long again.  In 64 bits it took 20 times as long."""
    m = require_gpu()
    z, b, _ = _inputs(65536, 256, 8, 0.05, std=1.5)
    z, b = _dev(z), _dev(b)
    opts = dict(score=kind, groups=groups, top_groups=top_groups)
    plain = _time(lambda: m.mxg_route_scores_fwd(z, 8, bias=b, **opts))
    for value in (-1e3, -1e9, -float(np.finfo(np.float32).max), 1e4, float("inf")):
        b2 = b.clone()
        b2[100] = value
        assert _time(lambda: m.mxg_route_scores_fwd(z, 8, bias=b2, **opts)) <= 1.5 * plain, value


# More tokens than the warps of a full grid take at once (456 blocks of 8 warps, 4 tokens each, 16 at 16 experts and 32 at
# 8), so that every warp takes several sets and one that is not whole.
SETS = [   # T, E, k, kind, bias, groups, top_groups, group_top, renormalize, scale
    (40001, 256, 8, "sigmoid", 0.05, 8, 4, 2, True, 2.5),
    (40001, 256, 8, "softmax", 0.002, 1, 1, 1, True, 1.0),
    (37003, 240, 6, "sigmoid", 0.05, 12, 5, 2, False, 1.0),     # groups across lanes
    (40001, 64, 8, "sigmoid", 0.05, 8, 4, 1, True, 1.0),
    (44449, 64, 32, "softmax", 0.01, 1, 1, 1, False, 1.0),
    (40001, 60, 4, "softmax", None, 10, 3, 2, True, 1.0),       # groups across lanes
    (50001, 64, 8, "softmax", None, 1, 1, 1, True, 1.0),        # by logits
    (150001, 16, 4, "sigmoid", 0.05, 2, 1, 2, True, 1.0),
    (300007, 8, 2, "sigmoid", 0.1, 4, 2, 2, True, 1.0),
]


@pytest.mark.parametrize("case", SETS, ids=[f"{c[0]}x{c[1]}{c[3]}g{c[5]}" for c in SETS])
def test_route_fwd_several_sets_to_a_warp(case):
    """Tokens that fp32 cannot decide stand in the first, the middle and the last sets, alone and side by side."""
    m = require_gpu()
    T, E, k, kind, bias = case[:5]
    z, b, rng = _inputs(T, E, k, bias, seed=5, std=1.5)
    at = np.unique(np.concatenate([np.arange(3), np.arange(T - 3, T), np.arange(T // 2, T // 2 + 9),
                                   rng.choice(T, T // 50, replace=False)]))
    near = (0.25 + rng.integers(0, 4, (at.size, E)) * np.float32(2.0 ** -24)).astype(np.float32)
    near[::5] = np.where(rng.random((near[::5].shape)) < 0.7, -np.inf, z[at[::5]])      # masked ones among them
    near[1::5, k // 2:] = z[at[1::5], k // 2:]                                           # a few that are close
    z[at] = near
    _check(m, z, b, k, _options(case))
