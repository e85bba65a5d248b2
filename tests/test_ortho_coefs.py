"""The limits of the orthogonalisation's coefficients (no GPU): they hold over the
whole interval that singular values can be in, also where a polynomial is at its
largest only within a narrow range, and calls on either side of them."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_matrix_host import AL, build, matrix  # noqa: E402
from zero_sharded_mixed_partition_amd import _lib as L  # noqa: E402


@pytest.fixture(scope="module")
def refused():
    _, buf = build([matrix()])
    d = AL - (1 << 30)

    def call(*steps):
        flat = [x for s in steps for x in s]
        # no room for the workspace: what passes the coefficients' check ends there
        st = L.lib().zero_multi_orthogonalize(buf, d, (ctypes.c_double * len(flat))(*flat), len(steps), 1e-7, None, d, 0, None)
        assert st in (L.ZERO_ENOSPC, L.ZERO_ERANGE), st
        return st == L.ZERO_ERANGE
    return call


def largest(a, b, c, top):
    """(of x (a + b x^2 + c x^4), of the polynomials), on [0, top]."""
    def extremes(p, ends):
        roots = p.deriv().roots() if p.degree() > 0 else []
        inside = [r.real for r in np.atleast_1d(roots) if abs(r.imag) < 1e-12 and ends[0] < r.real < ends[1]]
        return max(abs(p(x)) for x in (*ends, *inside))
    f = np.polynomial.Polynomial
    return (extremes(f([0, a, 0, b, 0, c]), (0, top)),
            max(extremes(f([0, b, c]), (0, top * top)), extremes(f([a, b, c]), (0, top * top))))


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("excess", [1e-4, 2e-8])
def test_either_side_of_the_limits(refused, seed, excess):
    """Random steps, scaled until one of their two largest values is at its limit."""
    rng = np.random.default_rng(seed)
    for k in range(20):
        tops = ((), ((0.3, 0.0, 0.0),), ((0.125, 0.0, 0.0),), ((1.5, -0.5, 0.0),))[k % 4]
        top = (1.0, 0.3, 0.125, 1.0)[k % 4]
        step = rng.normal(size=3) * (1.0, top ** -2, top ** -4)
        if k % 5 == 0:
            step[rng.integers(3)] = 0.0
        if k % 7 == 0:
            step[:] = 0.0, step[1], -step[1] / top ** 2 * rng.uniform(0.5, 0.95)
        if not step.any():
            continue
        x, p = largest(*step, top)
        by = min(4.0 / x, 32.0 / p)
        if by == 32.0 / p and x * by < 0.0625:
            continue
        assert not refused(*tops, step * by * (1 - excess)), (step, tops)
        assert refused(*tops, step * by * (1 + excess)), (step, tops)


def test_a_peak_between_samples(refused):
    """b y + c y^2 at its largest 5e-7 above the limit, within 1e-5 of x^2 = 1 / 128."""
    first = (0.125, 0.0, 0.0)
    for peak, out in ((32 - 5e-7, False), (32 + 5e-7, True)):
        b = 2 * peak * 128
        assert refused(first, (0.0, b, -b * 64)) == out


def test_extreme_coefficients(refused):
    for step in ((0.0, 1e308, -1e308), (0.0, 1e200, -1e200), (1e308, 0.0, 0.0), (1.0, 0.0, 1e308), (1.0, -1e308, 0.0),
                 (0.0, 1e308, 1e-308), (1e-300, 1e-300, 1e-300)):
        assert refused(step), step
    assert not refused((1.0, 1e-320, -1e-320)) and not refused((1.0, 0.0, -1e-300)) and not refused((-1.0, -0.0, 0.0))


@pytest.mark.parametrize("kind", [list, tuple, iter, lambda x: (s for s in x)])
def test_the_binding_counts_each_step(kind):
    """Also of steps that can be gone through only once: three of two numbers are not two of three."""
    import zero_sharded_mixed_partition_amd as Z
    with pytest.raises(ValueError, match="three numbers"):
        Z.zero_multi_orthogonalize(None, None, coefs=kind([(1.5, -0.5)] * 3))
