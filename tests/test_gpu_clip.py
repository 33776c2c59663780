"""Norm over all gradients and clipping on the GPU against the fp64 oracle."""
import numpy as np
import pytest
import torch

from gpu_helpers import np_, require_gpu
from oracle import block

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B = 2.0 ** -8
# a thread's squares of a chunk in fp32: a chain of 8 in a 16-byte piece, of 8 pieces, and a last single one, each square
# rounded in its fma, all under a root; the rest is fp64 and rounded once
NORM = (8 + 8 + 1) / 2 * U + 2 * U
SINGLY = 64 / 2 * U + 2 * U   # memory that starts on no 16 bytes: a chain of 64
SETS = {
    "one": [(1,)],
    "short": [(3,), (1, 1), (7, 5)],
    "ragged": [(16383,), (16384,), (16385,), (2, 8192), (8,), (100003,)],
    "layer": [(128,), (4, 128), (4, 512, 128), (4, 128, 256)],
    "empty among": [(0,), (300,), (4, 0, 7), (17,), (0, 3)],
    "many": [(i % 41 + 1,) for i in range(40)],
    "over one table": [(i % 5 + 1,) for i in range(1100)],
    "long": [(3000001,), (5,), (1 << 20,)],
}


def _grads(shapes, seed=0, std=0.01):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * std * (1 + i % 3)).to(torch.bfloat16 if i % 2 else torch.float32)
            for i, s in enumerate(shapes)]


def _check(got, grads, norm, most, tol=NORM):
    coef = min(1.0, most / norm) if norm else 1.0
    for a, g in zip(got, grads):
        ref = g.double().numpy() * coef
        rel = 0.0 if coef == 1.0 else tol + 3 * U + (U if g.dtype == torch.float32 else B)
        assert a.dtype == g.dtype and (np.abs(np_(a.double()) - ref) <= rel * np.abs(ref) + 1e-44).all()


@pytest.mark.parametrize("name", SETS)
def test_clip(name):
    m = require_gpu()
    grads = _grads(SETS[name])
    dev = [g.cuda() for g in grads]
    ref = block.grad_norm([g.double().numpy() for g in grads])
    assert abs(float(m.mxg_grad_norm(dev)) - ref) <= NORM * ref
    for most in (0.5 * ref, 2.0 * ref):
        out = [torch.full_like(g, 7.0) for g in dev]
        norm, got = m.mxg_grad_clip(dev, most, out=out)
        assert got is out and abs(float(norm) - ref) <= NORM * ref
        assert all(torch.equal(d.cpu(), g) for d, g in zip(dev, grads))
        _check(got, grads, ref, np.float32(most))
        again = m.mxg_grad_clip(dev, most, out=[torch.empty_like(g) for g in dev])
        assert torch.equal(again[0], norm) and all(torch.equal(a, b) for a, b in zip(again[1], got))
        here = [d.clone() for d in dev]
        norm2, got2 = m.mxg_grad_clip(here, most)
        assert got2 is here and torch.equal(norm2, norm) and all(torch.equal(a, b) for a, b in zip(got2, got))
        # by a norm that was taken before
        got3 = m.mxg_grad_clip(dev, most, out=[torch.empty_like(g) for g in dev], norm=norm)[1]
        _check(got3, grads, ref, np.float32(most))


@pytest.mark.parametrize("offset", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_any_element_address(dtype, offset):
    m = require_gpu()
    g = torch.Generator().manual_seed(offset)
    flat = torch.randn(50000, generator=g).to(dtype)
    views = [(offset, 40001), (40001 + offset, 9), (45000, 4999)]
    dev, out = flat.cuda(), torch.full((50000,), 7.0, dtype=dtype, device="cuda")
    grads = [flat[a:a + n] for a, n in views]
    norm, got = m.mxg_grad_clip([dev[a:a + n] for a, n in views], 3.0, out=[out[a:a + n] for a, n in views])
    ref = block.grad_norm([v.double().numpy() for v in grads])
    assert abs(float(norm) - ref) <= SINGLY * ref
    _check(got, grads, ref, 3.0, SINGLY)
    rest = torch.ones(50000, dtype=torch.bool, device="cuda")
    for a, n in views:
        rest[a:a + n] = False
    assert bool((out[rest] == 7.0).all())                 # what lies between is left as it was


@pytest.mark.parametrize("size", [1e-44, 1e-40, 1e-30, 1e-20, 1e19, 1e30, 1e36, 1e37])
def test_any_size(size):
    """Squares that leave fp32's range."""
    m = require_gpu()
    rng = np.random.default_rng(3)
    a = torch.from_numpy((rng.standard_normal(70001) * size).astype(np.float32))
    b = a[:999].bfloat16()
    zero = torch.zeros(5000)
    ref = block.grad_norm([a.double().numpy(), b.double().numpy()])
    with np.errstate(over="ignore"):
        most = float(np.float32(ref / 3))
    norm, got = m.mxg_grad_clip([a.cuda(), b.cuda(), zero.cuda()], most,
                                out=[torch.empty_like(t).cuda() for t in (a, b, zero)])
    tiny = 2.0 ** -149                                    # a norm among the numbers below fp32's normal ones
    if ref > 3.5e38:                                      # 70001 values of 1e37: the norm itself is beyond fp32
        assert float(norm) == float("inf") == float(m.mxg_grad_norm([a.cuda()]))
        _check(m.mxg_grad_clip([a.cuda()], 1e30, out=[torch.empty_like(a).cuda()])[1], [a],
               block.grad_norm([a.double().numpy()]), np.float32(1e30))
        return
    assert abs(float(norm) - ref) <= NORM * ref + tiny
    if size > 1e-36:
        _check(got, [a, b, zero], ref, most)
    mixed = [a.cuda(), torch.full((20000,), 1.0, device="cuda")]
    both = block.grad_norm([a.double().numpy(), np.ones(20000)])
    assert abs(float(m.mxg_grad_norm(mixed)) - both) <= NORM * both


def test_zero_infinite_and_nan():
    m = require_gpu()
    z = [torch.zeros(1000, device="cuda"), torch.zeros(3, 7, dtype=torch.bfloat16, device="cuda")]
    norm, got = m.mxg_grad_clip(z, 1.0, out=[torch.ones_like(t) for t in z])
    assert float(norm) == 0.0 and not got[0].any() and not got[1].any()
    z = [torch.empty(0, device="cuda")]
    assert float(m.mxg_grad_norm(z)) == 0.0 and float(m.mxg_grad_clip(z, 1.0)[0]) == 0.0
    a = torch.ones(20000, device="cuda")
    a[17] = float("inf")
    norm, (got,) = m.mxg_grad_clip([a], 1.0, out=[torch.ones_like(a)])
    assert float(norm) == float("inf") and bool(got[17].isnan()) and int((got == 0).sum()) == 19999
    a[17] = float("nan")
    norm, (got,) = m.mxg_grad_clip([a], 1.0, out=[torch.ones_like(a)])
    assert bool(norm.isnan()) and bool(got.isnan().all())
    norm, (got,) = m.mxg_grad_clip([torch.ones(4, device="cuda")], float("inf"))
    assert float(norm) == 2.0 and bool((got == 1.0).all())


def test_same_output_twice_is_refused():
    m = require_gpu()
    a, b = torch.ones(40, device="cuda"), torch.ones(40, device="cuda")
    with pytest.raises(ValueError, match="twice"):
        m.mxg_grad_clip([a, b, a], 1.0)
    with pytest.raises(ValueError, match="twice"):
        m.mxg_grad_clip([a, b], 1.0, out=[a, a])
    assert abs(float(m.mxg_grad_norm([a, a])) - 80 ** 0.5) <= NORM * 9
    with pytest.raises(ValueError, match="contiguous"):
        m.mxg_grad_norm([torch.ones(4, 4, device="cuda").t()[1:]])


@pytest.mark.parametrize("size,most", [(1e35, 1e-3), (1e35, 1e-12), (1e37, 1.0), (1e37, 1e-20), (1e37, 1e-28), (1e30, 1e-25),
                                       (1e20, 1e-25)])
def test_factors_below_normal_numbers(size, most):
    """max_norm / norm below what fp32 holds in full (2^-126, or nothing left at 2^-150), whose products fp32 holds."""
    m = require_gpu()
    rng = np.random.default_rng(4)
    a = torch.from_numpy((rng.uniform(-3.0, 3.0, 70001) * size).astype(np.float32))
    b = a[:999].bfloat16()
    ref = block.grad_norm([a.double().numpy(), b.double().numpy()])
    most = np.float32(most)
    norm, got = m.mxg_grad_clip([a.cuda(), b.cuda()], float(most), out=[torch.empty_like(t).cuda() for t in (a, b)])
    _check(got, [a, b], ref, np.float64(most))
    if ref < 3e38:                                        # by the norm that was taken before
        got = m.mxg_grad_clip([a.cuda(), b.cuda()], float(most), out=[torch.empty_like(t).cuda() for t in (a, b)], norm=norm)[1]
        _check(got, [a, b], ref, np.float64(most))


def test_an_output_is_no_other_gradient():
    """The scaling pass would read a gradient that other blocks have overwritten."""
    m = require_gpu()
    a, b, c = torch.full((40,), 1.0, device="cuda"), torch.full((40,), 2.0, device="cuda"), torch.empty(40, device="cuda")
    none = torch.empty(0, device="cuda")
    for grads, out in (([a, b], [b, a]), ([a, b], [b, c]), ([a, b], [c, a]), ([a, a], [a, c])):
        with pytest.raises(ValueError, match="gradient"):
            m.mxg_grad_clip(grads, 1.0, out=out)
        with pytest.raises(ValueError, match="gradient"):
            m.mxg_grad_clip(grads, 1.0, out=out, norm=torch.ones(1, device="cuda"))
    assert bool((a == 1.0).all()) and bool((b == 2.0).all())
    norm, out = m.mxg_grad_clip([a, none, b], 1.0, out=[a, torch.empty(0, device="cuda"), c])     # some in place
    _check([out[0], out[2]], [torch.full((40,), 1.0), torch.full((40,), 2.0)], 200 ** 0.5, 1.0)
    assert abs(float(norm) - 200 ** 0.5) <= NORM * 200 ** 0.5


def test_outputs_of_another_shape():
    """An output takes its gradient's elements in the order of the memory: views of one flat buffer, as buckets are."""
    m = require_gpu()
    grads = [g.cuda() for g in _grads([(6, 4), (5,), (3, 2, 7)])]
    ref = m.mxg_grad_clip(grads, 0.01, out=[torch.empty_like(g) for g in grads])[1]
    flat = {t: torch.full((71,), 7.0, dtype=t, device="cuda") for t in (torch.float32, torch.bfloat16)}
    out = [flat[grads[0].dtype][:24], flat[grads[1].dtype][:5], flat[grads[2].dtype][24:66]]
    got = m.mxg_grad_clip(grads, 0.01, out=out)[1]
    assert all(torch.equal(a, b.view(-1)) for a, b in zip(got, ref))
    assert bool((flat[grads[0].dtype][66:] == 7.0).all())
    for bad in (torch.empty(23, dtype=grads[0].dtype, device="cuda"), torch.empty(0, dtype=grads[0].dtype, device="cuda")):
        with pytest.raises(ValueError, match="24 elements"):
            m.mxg_grad_clip(grads, 0.01, out=[bad, *out[1:]])
