"""Clipping by the global norm on the GPU against 64-bit arithmetic: sizes
from none to more than 2^31 values, mixed types, unaligned tensors, more
tensors than one launch takes, values whose squares leave fp32's range, and
values that are not finite.

Bounds: the norm is within 2^-22 of its value (fp32 sums of at most 32
squares, then fp64: 32 roundings of 2^-24 at most, halved by the root, and
the last rounding); each output within half a step of its type of g c, with
c off by 2^-22 as the norm is and rounded to fp32, and the fp32 product
rounded once more."""
import math

import numpy as np
import pytest
import torch

import ffn_ref as ref

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ff():
    from hierarchical_gemm_gb300 import tsffn
    return tsffn


def _check(ff, grads, max_norm, in_place=False):
    g64 = [ref.f64(g) for g in grads]
    n, c = ref.clip(g64, max_norm)
    if in_place:
        out = grads
        norm = ff.clip_grad_norm(grads, max_norm)
    else:
        keep = [g.clone() for g in grads]
        out = [torch.full_like(g, float("nan")) for g in grads]
        norm = ff.clip_grad_norm(grads, max_norm, out=out)
    torch.cuda.synchronize()
    assert abs(float(norm) - n) <= 2.0 ** -22 * n
    for i, (o, g) in enumerate(zip(out, g64)):
        want = g * c
        ref.check(o, (want, ref.rounded(want, 2.0 ** -21 * np.abs(want), o.dtype)), "tensor %d" % i)
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(keep, grads))


def _tensors(sizes, kinds, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [torch.randn(n, generator=g, device="cuda").mul_(scale).to(kinds[i % len(kinds)])
            for i, n in enumerate(sizes)]


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("sizes", [[1], [7, 8, 9], [0, 5, 0], [8191, 8192, 8193, 1], [100000, 3, 250001]])
def test_sizes(ff, sizes, in_place, max_norm):
    for kinds in ([BF], [HF], [FL], [BF, FL, HF]):
        _check(ff, _tensors(sizes, kinds, 1), max_norm, in_place)


def test_no_tensors(ff):
    assert float(ff.clip_grad_norm([], 1.0)) == 0.0
    assert float(ff.clip_grad_norm([torch.empty(0, device="cuda")], 1.0)) == 0.0
    z = [torch.zeros(1000, dtype=BF, device="cuda")]
    assert float(ff.clip_grad_norm(z, 1.0)) == 0.0 and bool((z[0] == 0).all())


def test_many_tensors(ff):
    # more than one launch takes
    _check(ff, _tensors([(i * 37) % 300 for i in range(1300)], [BF, FL, HF], 2), 0.25)
    _check(ff, _tensors([11] * 513, [BF], 3), 0.25, in_place=True)


def test_unaligned(ff):
    base = _tensors([5000, 5000, 5000], [BF, FL, HF], 4)
    views = [b[1:1 + n] for b, n in zip(base, (999, 4097, 12))] + [base[0][1003:1500], base[1][4201:4202]]
    edges = [(b[0].clone(), b[-1].clone()) for b in base]
    _check(ff, views, 0.5)
    _check(ff, views, 0.5, in_place=True)
    assert all(torch.equal(b[0], e[0]) and torch.equal(b[-1], e[1]) for b, e in zip(base, edges))


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-22, 1e-18, 1e17, 1e19, 1e25, 1e35])
def test_squares_outside_fp32(ff, scale):
    for kinds in ([FL], [BF], [BF, FL]):
        # (1e-42: below fp32's normal range, where a value itself has few bits)
        grads = _tensors([3000, 41], kinds, 5, scale)
        n, _ = ref.clip([ref.f64(g) for g in grads], 1.0)
        norm = float(ff.clip_grad_norm(grads, math.inf, out=[torch.empty_like(g) for g in grads]))
        assert abs(norm - n) <= 2.0 ** -22 * n + 2.0 ** -150
        if 1e-10 * scale > 1e-37 and n < 1e38:
            _check(ff, grads, n / 3)
    mixed = torch.cat([t.float() for t in _tensors([500, 500, 500], [FL], 6)])
    mixed[:500] *= 1e30
    mixed[500:1000] *= 1e-30
    _check(ff, [mixed], 1.0)


def test_a_lone_large_value_among_small(ff):
    for big in (1e20, 1e30):
        x = torch.full((20000,), 1e-3, device="cuda")
        x[12345] = big
        _check(ff, [x], 1.0)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_not_finite(ff, bad):
    # the formula's own course: a norm that is inf gives a coefficient of 0
    # (and inf * 0 is a NaN), one that is NaN gives NaN everywhere
    x = torch.ones(9000, dtype=BF, device="cuda")
    x[4321] = bad
    out = torch.empty_like(x)
    norm = float(ff.clip_grad_norm([x], 1.0, out=[out]))
    if math.isnan(bad):
        assert math.isnan(norm) and bool(torch.isnan(out).all())
    else:
        assert norm == math.inf and bool(torch.isnan(out[4321])) and float(out.float().nan_to_num().abs().max()) == 0.0


def test_below_the_limit_nothing_changes(ff):
    g = _tensors([1000, 77], [BF, FL], 7)
    keep = [t.clone() for t in g]
    ff.clip_grad_norm(g, 1e6)
    assert all(torch.equal(a, b) for a, b in zip(g, keep))


def test_the_norm_alone(ff):
    # no limit: nothing changes, not even for a norm that is not finite
    for extra in (0.0, math.inf, math.nan):
        g = _tensors([1000, 77], [BF, FL], 9)
        g[0][3] = extra
        keep = [t.clone() for t in g]
        norm = float(ff.clip_grad_norm(g, math.inf))
        assert math.isfinite(norm) == math.isfinite(extra)
        assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(g, keep))


def test_reproducible(ff):
    g = _tensors([1234567, 4097, 3], [BF, FL, HF], 8)
    one = float(ff.clip_grad_norm(g, 1.0, out=[torch.empty_like(t) for t in g]))
    for _ in range(5):
        assert float(ff.clip_grad_norm(g, 1.0, out=[torch.empty_like(t) for t in g])) == one


def test_more_than_32_bits_of_values(ff):
    n = (1 << 31) + 12345
    x = torch.zeros(n, dtype=BF, device="cuda")
    x[:1000] = 1.0
    x[-1000:] = 2.0
    norm = float(ff.clip_grad_norm([x], 1.0))
    want = math.sqrt(5000.0)
    assert abs(norm - want) <= 2.0 ** -22 * want
    c = 1.0 / (want + 1e-6)
    assert abs(float(x[-1]) - 2 * c) <= 2.0 ** -8 * 2 * c and abs(float(x[0]) - c) <= 2.0 ** -8 * c
    assert float(x[n // 2]) == 0.0
