"""Polynomials with a coefficient far below the others: their largest value is
inside the range of the singular values, and the number formats have to hold
it."""
import pytest
import torch

import optimizer_step_layeradam_amd as la
from muonhelpers import H, HALF_STEP, direction64, matrices, off

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(40, 90), (3, 7), (200, 170)])
@pytest.mark.parametrize("c", [0.0, 1e-17, -1e-17, 1e-15])
def test_largest_value_inside_the_range(c, shape):
    """3 s - 2.99 s^3 is 1.157 at 3^-1/2, where three equal singular values lie,
    and 0.01 at 1. The three are rounded alike, so roundings add up rather than
    average: h = 2^-11 at most for X as the products read it, three times in the
    first step's b A X, |b| l / (a + b l) = 0.997 / 2.003 of the result each: 1.5 h.
    The second step reads X with that and a rounding of its own, and its slope
    s p'(s) / p(s) at 1.157 is 3 - 3 * 2.99 * 1.339 = -9.0: 9 (1 + 1.5) h = 22.5 h. What
    lies beside the three is ten thousand times smaller."""
    x = matrices(shape, seed=3, scale=1e-4)
    x[0, 0] = x[1, 1] = x[2, 2] = 1.0
    steps = ((3.0, -2.99, c),) * 2
    o = la.orthogonalize(x.cuda(), torch.empty(shape, dtype=torch.float16, device="cuda"),
                         coefficients=steps)
    got = off(o, direction64(x, steps))
    print(f"  {shape} c = {c}: off {got:.2e}", flush=True)
    assert got <= 23 * H + HALF_STEP[torch.float16]
