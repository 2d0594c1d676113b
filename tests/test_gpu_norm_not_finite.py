"""The norms over rows that hold infinities, and over rows whose squares pass the
range of FP32: what each result is there, and that the rows beside keep theirs.
Exact: zeros, NaN and the bias itself. Rows of every kernel: in the registers of
4 to 1024 lanes, of 1024 alone, and read once a sum."""
import pytest
import torch

import optimizer_step_layeradam_amd as la
from normhelpers import inputs, params

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
COLS = [5, 100, 1030, 8192, 12288, 20000, 33000]
INF = float("inf")


def problem(cols, dtype):
    x, dy, ds = (inputs(6, cols, dtype, k).cuda() for k in (1, 2, 3))
    w, b = (t.cuda() for t in params(cols, F, 4))
    return x, dy, ds, w, b


def both(layer, x, dy, ds, w, b):
    if layer:
        y, stats = la.layer_norm(x, w, b)
        return (y, stats, *la.layer_norm_backward(dy, x, w, stats, residual_grad=ds))
    y, stats = la.rms_norm(x, w)
    return (y, stats, *la.rms_norm_backward(dy, x, w, stats, residual_grad=ds), None)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("bad", [INF, -INF])
def test_infinities(layer, cols, dtype, bad):
    x, dy, ds, w, b = problem(cols, dtype)
    want = both(layer, x, dy, ds, w, b)
    at = cols // 2
    x[3, at] = bad
    y, stats, dx, dw, db = both(layer, x, dy, ds, w, b)
    keep = [0, 1, 2, 4, 5]
    for got, e in ((y, want[0]), (dx, want[2])):
        assert torch.equal(got[keep], e[keep])
    assert torch.equal(stats[:, keep], want[1][:, keep])
    others = torch.arange(cols, device="cuda") != at
    assert bool(y[3, at].isnan()) and bool(dx[3].isnan().all()) and bool(dw[at].isnan())
    if layer:
        assert bool(y[3].isnan().all()) and bool(stats[1, 3].isnan()) and bool(dw.isnan().all())
        assert torch.equal(db, want[4])  # x is no part of it
    else:
        assert float(stats[0, 3]) == 0.0 and bool((y[3, others] == 0).all())
        assert bool(dw[others].isfinite().all())


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("layer", [True, False])
def test_squares_past_the_range(layer, cols, dtype):
    x, dy, ds, w, b = problem(cols, dtype)
    zeroed = x.clone()
    want = both(layer, x, dy, ds, w, b)
    # 2^100 and -2^100 in turn: squares of 2^200, sums that any order keeps below 2^116
    x[3] = 2.0 ** 100
    x[3, ::2] = -2.0 ** 100
    y, stats, dx, dw, db = both(layer, x, dy, ds, w, b)
    keep = [0, 1, 2, 4, 5]
    for got, e in ((y, want[0]), (dx, want[2])):
        assert torch.equal(got[keep], e[keep])
    assert float(stats[-1, 3]) == 0.0
    assert torch.equal(y[3], b.to(dtype) if layer else torch.zeros_like(y[3]))
    assert torch.equal(dx[3], ds[3])
    # dweight is that of the other rows: rows of zeros with a rstd of 0 add as little
    if layer:
        assert torch.equal(db, want[4])
    stats0 = want[1].clone()
    stats0[-1, 3] = 0.0
    if layer:
        stats0[0, 3] = 0.0
    zeroed[3] = 0.0
    back = la.layer_norm_backward if layer else la.rms_norm_backward
    assert torch.equal(back(dy, zeroed, w, stats0, residual_grad=ds)[1], dw)
