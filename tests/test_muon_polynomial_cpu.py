"""Which polynomials the library takes, by their largest value on the range of
the singular values. Host only."""
import pytest

import optimizer_step_layeradam_amd as la

SHAPES = [(300, 400)]


def taken(*steps):
    try:
        return la.orthogonalize_workspace_bytes(SHAPES, coefficients=steps) > 0
    except la.LayerAdamError:
        return False


@pytest.mark.parametrize("c", [0.0, 1e-300, 1e-20, -1e-20, 1e-17, -1e-17, 1e-15, -1e-15, 1e-9])
def test_inner_extreme_beside_a_tiny_coefficient(c):
    # 0 at s = 1, 0.77 at s = 3^-1/2: the largest value is an inner one
    assert taken((2.0, -2.0, c))
    # 1 at s = 1, 1.6e6 > 2^20 inside
    assert not taken((2.0 ** 22, 1.0 - 2.0 ** 22, c))


def test_bounds_against_a_grid():
    """The refusal's border, 2^20, against the largest value on a grid of the
    range: polynomials scaled to end on either side of it."""
    grid = [i / 4000 for i in range(4001)]
    shapes = [(a, b, c) for a in (3.0, -1.0, 0.5, 0.0) for b in (-4.0, 2.5, 1e-18, 0.0)
              for c in (2.0, -1.5, 1e-17, -1e-17, 0.0)]
    for a, b, c in shapes:
        most = max(abs(a * x + b * x ** 3 + c * x ** 5) for x in grid)
        if most < 1e-6:
            continue
        # the grid misses the largest value by (1 / 8000)^2 / 2 of the curvature, at most
        # 100 times the coefficients: a part in a thousand is ample
        for f in (0.999, 1.001):
            k = f * 2.0 ** 20 / most
            assert taken((a * k, b * k, c * k)) == (f < 1.0), (a, b, c, f)
