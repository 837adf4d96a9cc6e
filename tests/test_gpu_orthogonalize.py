"""fsdp_orthogonalize over steps, polynomials and kinds of matrices against its
definition in 64 bits (products_ref).

Tolerances, in the 2-norm relative to the result. Rounding the result to
bfloat16: 2^-8 over the square root of 3, 2.3e-3. With more than 64 rows and
columns each step rounds four factors to binary16, which reaches the result as
2^-11 a step (test_gpu_products). With at most 64 rows or
columns X is held in binary32: a step leaves in each element an error of the
order of 2^-24 of the terms that it sums, (|a| + |b| + |c|) |X| / sqrt(p q) for
singular values near one at most, and errors of elements that are independent
have singular values of at most (sqrt(p) + sqrt(q)) of theirs. A direction in
which x has a singular value s sees that relative to s / |x|; the steps lift
both alike, and those after the first, whose X has grown, add less than half of
what the steps before them added. Four times that is allowed for."""
import math

import pytest
import torch

import products_ref as R
from hsdp_sharded_parameter_gb300 import capi as C
from test_gpu_products import BF16, F32, matrix, no_wait_ran_out, ortho  # noqa: F401

pytestmark = pytest.mark.gpu

DEFAULT, CUBIC, QUINTIC = (3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)
ROUNDED = 2.3e-3
HELD_IN_16_BITS = ROUNDED + 5 * 2.0 ** -11  # five steps


def held_in_32_bits(x, coefficients):
    s = torch.linalg.svdvals(R.d(x))
    p, q = min(x.shape), max(x.shape)
    spread = float(s.square().sum().sqrt() / s.min())
    return ROUNDED + 4 * sum(map(abs, coefficients)) * 2.0 ** -24 * (p ** 0.5 + q ** 0.5) / (p * q) ** 0.5 * spread


@pytest.mark.parametrize("steps, coefficients", [(7, DEFAULT), (8, DEFAULT), (9, DEFAULT), (12, DEFAULT), (16, QUINTIC), (24, QUINTIC), (40, QUINTIC),
                                                 (25, CUBIC), (30, CUBIC), (64, CUBIC)])
@pytest.mark.parametrize("rows, cols", [(64, 200), (200, 64), (33, 70), (12, 3000)])
def test_few_rows_over_many_steps(rows, cols, steps, coefficients):
    for kind in ("noise", "low"):
        x = matrix(kind, rows, cols, F32)
        got = ortho(x, steps=steps, coefficients=coefficients)
        assert R.distance(got, R.orthogonalize(x, steps, coefficients)) < held_in_32_bits(x, coefficients)


@pytest.mark.parametrize("steps, coefficients, most", [(5, DEFAULT, 1.21), (10, DEFAULT, 1.21), (30, DEFAULT, 1.21), (64, DEFAULT, 1.21), (24, QUINTIC, 1.0),
                                                       (64, QUINTIC, 1.0), (40, CUBIC, 1.0)])
@pytest.mark.parametrize("rows, cols", [(8, 512), (64, 1024), (1024, 64)])
def test_matrices_without_full_rank_stay_bounded(rows, cols, steps, coefficients, most):
    # rows that repeat: the rank is 2, exactly. In the other directions there is what rounding
    # leaves, which the steps lift as they lift anything else: the polynomials map [0, most] into itself.
    few, many = min(rows, cols), max(rows, cols)
    base, which = matrix("noise", 2, many, F32), torch.arange(few, device="cuda") % 2
    x = base[which].contiguous()
    got = R.d(ortho(x if rows <= cols else x.t().contiguous(), steps=steps, coefficients=coefficients))
    got = got if rows <= cols else got.T
    # rounding to bfloat16 moves singular values by its norm, ROUNDED of |out|, at most
    slack = ROUNDED * float(got.norm()) + 1e-3
    assert bool(torch.isfinite(got).all())
    assert float(torch.linalg.eigvalsh(got @ got.T).max().sqrt()) < most + slack
    if coefficients != DEFAULT:
        # x = U (D base) with U's columns orthonormal, and these polynomials bring D base to its nearest orthonormal rows
        U = (which.cpu()[:, None] == torch.arange(2)) / (few / 2) ** 0.5
        s, v = torch.linalg.eigh(R.d(base) @ R.d(base).T)
        nearest = v @ torch.diag(s ** -0.5) @ v.T @ R.d(base)
        assert float((U.double().T @ got - nearest).norm()) < slack


@pytest.mark.parametrize("rows, cols", [(64, 3000), (1000, 1000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("std", [1e-43, 1e-40, 1e-37, 1e-25, 1e-13, 1e-12, 1e15, 2e15, 5e17, 3e18, 1e36, 5e37])
def test_any_finite_values(rows, cols, dtype, std):
    # the sums of squares of these reach from 2^-290 to 2^270. A value of 1e-43 is up to 71 steps of the
    # smallest one of float32, and none of bfloat16.
    if dtype == BF16 and std < 1e-40:
        return
    x = matrix("noise", rows, cols, dtype, std=std)
    assert bool(torch.isfinite(x).all()) and bool(x.any())
    assert R.distance(ortho(x, eps=0.0), R.orthogonalize(x, eps=0.0)) < HELD_IN_16_BITS


@pytest.mark.parametrize("rows, cols", [(40, 70), (100, 130), (130, 100)])
def test_one_large_value_among_small_ones(rows, cols):
    x = matrix("noise", rows, cols, F32, std=1e-20)
    x[3, 5] = 3e38
    got = ortho(x, eps=0.0)
    assert R.distance(got, R.orthogonalize(x, eps=0.0)) < HELD_IN_16_BITS


@pytest.mark.parametrize("rows, cols", [(100, 130), (130, 100), (300, 300)])
def test_infinities_and_nan(rows, cols):
    for bad in (math.inf, -math.inf, math.nan):
        x = matrix("noise", rows, cols, F32).clone()
        x[7, 9] = bad
        assert bool(torch.isnan(ortho(x)).all())
    assert not bool(ortho(torch.zeros(rows, cols, device="cuda")).any())


@pytest.mark.parametrize("rows, cols", [(40, 70), (100, 130)])
@pytest.mark.parametrize("eps", [5e-324, 1e-300, 1e-40, 1.0, 1e300])
def test_zeros_stay_zeros(rows, cols, eps):
    assert not bool(ortho(torch.zeros(rows, cols, device="cuda"), eps=eps).any())


def condition(x, steps, coefficients):
    """By how much, at most, an error of X is larger after the steps than before, both relative."""
    a, b, c = coefficients
    s = torch.linalg.svdvals(R.d(x) / R.d(x).norm())
    k = torch.ones_like(s)
    for _ in range(steps):
        p = a * s + b * s ** 3 + c * s ** 5
        k, s = k * (s * (a + 3 * b * s ** 2 + 5 * c * s ** 4) / p).abs(), p.abs()
    return max(1.0, float(k.max()))


@pytest.mark.parametrize("steps, coefficients", [(1, (256.0, 0.0, 0.0)), (2, (8.0, 0.0, 0.0)), (2, (-8.0, 0.0, 0.0)), (4, (2.0, 0.0, 0.0)), (3, (4.0, -6.0, 3.0)),
                                                 (2, (8.28721201814563, -23.595886519098837, 17.300387312530933)), (1, (256.0, -256.0, 256.0))])
@pytest.mark.parametrize("rows, cols", [(40, 70), (96, 200), (200, 96)])
def test_polynomials_that_grow(rows, cols, steps, coefficients):
    x = matrix("noise", rows, cols, F32)
    want = R.orthogonalize(x, steps, coefficients)
    assert R.distance(ortho(x, steps=steps, coefficients=coefficients), want) < ROUNDED + steps * 2.0 ** -11 * condition(x, steps, coefficients)


@pytest.mark.parametrize("rows, cols", [(40, 1100), (1100, 1100), (2100, 1100)])
def test_polynomials_that_grow_one_singular_value(rows, cols):
    # all of A is one value, 64 before the last step
    x = matrix("noise", rows, cols, F32, std=1e-6)
    x[30, 40] = 1.0
    want = R.orthogonalize(x, 2, (8.0, 0.0, 0.0))
    assert R.distance(ortho(x, steps=2, coefficients=(8.0, 0.0, 0.0)), want) < ROUNDED + 2 * 2.0 ** -11
    want = R.orthogonalize(x, 2, (4.0, 3.0, 1.0))
    assert R.distance(ortho(x, steps=2, coefficients=(4.0, 3.0, 1.0)), want) < ROUNDED + 2 * 2.0 ** -11 * 25  # of a fifth power twice


@pytest.mark.parametrize("steps, coefficients", [(1, DEFAULT), (5, DEFAULT), (40, QUINTIC), (3, (1.0, 0.0, 0.0)), (3, (0.25, 0.0, 0.0)), (2, (8.0, 0.0, 0.0))])
@pytest.mark.parametrize("rows, cols", [(40, 70), (100, 130), (1030, 520)])
@pytest.mark.parametrize("kind", ["noise", "spikes"])
def test_eps_far_above_the_norm(rows, cols, kind, steps, coefficients):
    # X_0 is x over eps, and small: what the steps leave of it is as exact as ever
    x = matrix(kind, rows, cols, F32)
    norm = float(R.d(x).norm())
    for ratio in (1e-2, 1.0, 1e2, 1e4, 1e7, 1e10, 1e15, 1e25):
        k = dict(steps=steps, coefficients=coefficients, eps=norm * ratio, scale=2.0)
        assert R.distance(ortho(x, **k), R.orthogonalize(x, **k)) < ROUNDED + steps * 2.0 ** -11, ratio


@pytest.mark.parametrize("shape", [(1, 30000001), (50000017, 1), (1, 1 << 25), (2, 10 ** 7)], ids=str)
def test_long_rows(shape):
    # a + b A leaves 1/16 of X, so an error of A shows 31 times as large. A's sum over a row is in stretches of at
    # most 2048 additions, and of less than 64 stretches a part at these lengths, so where all roundings go the
    # same way A is off by 2112 * 2^-24 at most.
    x = torch.ones(shape, device="cuda")
    if min(shape) > 1:
        x[1] = torch.randn(shape[1], generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 1e-6
    work = torch.empty(C.fsdp_orthogonalize_workspace(*shape), dtype=torch.uint8, device="cuda")
    out = torch.empty(shape, dtype=BF16, device="cuda")
    C.fsdp_orthogonalize(x, out, work, steps=1, coefficients=(2.0, -1.9375, 0.0))
    want = R.orthogonalize(x, 1, (2.0, -1.9375, 0.0))
    # the same rounding in all places, so no mean over places helps: half a step of bfloat16, which has 8 bits,
    # is 2^-8 of a value just above a power of two (1.1411e-5 = 191.45 steps of 2^-24 becomes 191 of them)
    assert R.distance(out, want) < 2.0 ** -8 + 31 * 2112 * 2.0 ** -24
