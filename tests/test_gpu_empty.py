"""The norms and the linear cross entropy on tensors without rows, in every
place of the axis that has none."""
import pytest
import torch

import optimizer_step_layeradam_amd as la

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("lead", [(0,), (2, 0), (0, 2), (2, 0, 3), (2, 3, 0), (5, 2, 0, 3)])
def test_no_rows(lead):
    w = torch.randn(500, 64, device="cuda").to(BF)
    x = torch.empty(*lead, 64, dtype=BF, device="cuda")
    y = torch.empty(lead, dtype=torch.int64, device="cuda")
    loss, dx, dw = la.linear_cross_entropy_gradients(x, w, y)
    assert float(loss) == 0.0 and dx.shape == x.shape and bool((dw == 0).all())
    dw.fill_(3)
    la.linear_cross_entropy_gradients(x, w, y, dx=dx, dweight=dw)
    assert bool((dw == 0).all())
    assert float(la.linear_cross_entropy(x, w, y, reduction="sum")) == 0.0

    gamma = torch.ones(64, device="cuda")
    out, stats, s = la.layer_norm(x, gamma, gamma, residual=x)
    assert out.shape == s.shape == x.shape and stats.shape == (2, 0)
    dx, dgamma, dbeta = la.layer_norm_backward(out, s, gamma, stats)
    assert dx.shape == x.shape and bool((dgamma == 0).all()) and bool((dbeta == 0).all())
    out, stats = la.rms_norm(x, gamma)
    dx, dgamma = la.rms_norm_backward(out, x, gamma, stats)
    assert dx.shape == x.shape and bool((dgamma == 0).all())


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("lead", [(1,), (5,), (2, 3, 4)])
def test_rows_without_elements(lead, given):
    """Means over nothing are NaN, and so are the statistics of such rows."""
    x = torch.empty(*lead, 0, dtype=BF, device="cuda")
    rows = torch.empty(lead).numel()
    for f, n in ((la.layer_norm, 2), (la.rms_norm, 1)):
        stats = torch.full((n, rows), 3.0, device="cuda") if given else None
        out, got = f(x, stats=stats)
        assert out.shape == x.shape and got.shape == (n, rows)
        want = torch.full((n, rows), float("nan"), device="cuda")
        if n == 2:  # as the plain form has them
            want[0] = x.float().mean(-1).reshape(-1)
        assert torch.equal(got.isnan(), want.isnan())
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        _, got = f(x, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert bool(got.isnan().all())
