"""Layer norm and RMS norm on the GPU against their formulas in 64 bits, to
bounds counted from their roundings (tests/normhelpers.py): every shape of the
kernels, types, strides, residuals, parameters left out, and what a call may
not do."""
import pytest
import torch

import optimizer_step_layeradam_amd as la
from normhelpers import (backward64, backward_bound, forward64, forward_bound, inputs, params,
                         within)

pytestmark = pytest.mark.gpu
BF, H, F = torch.bfloat16, torch.float16, torch.float32


def run(x, w, b, layer, eps, residual=None, dy=None, dsum=None, **kw):
    """Forward, and backward where dy is given; checked. All on the GPU."""
    norm = la.layer_norm if layer else la.rms_norm
    more = dict(bias=b) if layer else {}
    got = norm(x, w, eps=eps, residual=residual, **more, **kw)
    y, stats = got[:2]
    s = x
    if residual is not None:
        s = got[2]
        want = (x.float() + residual.float()).to(x.dtype)
        assert torch.equal(s.cpu(), want.cpu())
    assert y.dtype == x.dtype and y.shape == x.shape
    b = b if layer else None
    y64, mean64, rstd64 = forward64(s.cpu(), None if w is None else w.cpu(),
                                    None if b is None else b.cpu(), eps, layer)
    by, bm, br = forward_bound(s.cpu(), None if w is None else w.cpu(),
                               None if b is None else b.cpu(), eps, layer, y64, mean64, rstd64,
                               x.dtype)
    within(y, y64, by, "y")
    lead = x.shape[:-1]
    if layer:
        within(stats[0].reshape(lead), mean64, bm, "mean")
    within(stats[-1].reshape(lead), rstd64, br, "rstd")
    if dy is None:
        return got
    back = la.layer_norm_backward if layer else la.rms_norm_backward
    grads = back(dy, s, w, stats, residual_grad=dsum)
    mean = stats[0].reshape(lead).cpu() if layer else torch.zeros(lead)
    args = (dy.cpu(), s.cpu(), None if w is None else w.cpu(), mean, stats[-1].reshape(lead).cpu(),
            layer)
    want = backward64(*args, None if dsum is None else dsum.cpu())
    bounds = backward_bound(*args, *want, None if dsum is None else dsum.cpu(), x.dtype,
                            grads[1].dtype)
    for g, e, m, name in zip(grads, want, bounds, ("dx", "dweight", "dbias")):
        within(g, e, m, name)
    return got + tuple(grads)


SHAPES = [(1, 1), (3, 7), (9, 16), (70, 33), (257, 128), (33, 130), (5, 511), (1100, 96),
          (6, 1027), (7, 2560), (3, 4096), (5, 5120), (4, 6145), (3, 8192), (2, 8193), (3, 16384),
          (3, 16385), (2, 70001)]


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("dtype,wtype", [(BF, BF), (H, F), (F, F), (BF, F), (F, H)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_against_formulas(rows, cols, dtype, wtype, layer):
    x, dy = inputs(rows, cols, dtype, 1).cuda(), inputs(rows, cols, dtype, 2).cuda()
    w, b = (t.cuda() for t in params(cols, wtype))
    run(x, w, b, layer, 1e-5, dy=dy)


# Rows that fill the registers of 1024 lanes, from their shortest to their longest, whole
# vectors and not; more rows than workgroups, so that each adds rows up.
@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("added", [False, True])
@pytest.mark.parametrize("dtype,wtype,rows,cols", [
    (BF, BF, 3, 24576), (BF, F, 2, 24577), (BF, BF, 2, 32767), (H, H, 3, 32768), (H, F, 2, 16391),
    (F, F, 2, 8196), (F, H, 3, 12290), (F, F, 2, 16384), (F, BF, 2, 16387), (F, F, 3, 24576),
    (F, F, 2, 24579), (F, BF, 2, 32766), (F, F, 3, 32768), (BF, BF, 2, 32769), (F, F, 2, 32772),
    (BF, BF, 517, 16392), (F, F, 300, 8193)])
def test_wide_rows(dtype, wtype, rows, cols, added, layer):
    x, r, dy, ds = (inputs(rows, cols, dtype, k).cuda() for k in range(4))
    w, b = (t.cuda() for t in params(cols, wtype))
    if not added:
        r = ds = None
    run(x, w, b if layer else None, layer, 1e-5, r, dy, ds)


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("rows,cols", [(5, 100), (3, 2561), (4, 20000)])
def test_residual(rows, cols, dtype):
    x, r, dy, ds = (inputs(rows, cols, dtype, k).cuda() for k in range(4))
    w, b = (t.cuda() for t in params(cols, dtype))
    run(x, w, b, True, 1e-5, r, dy, ds)
    run(x, w, None, False, 1e-6, r, dy, ds)
    run(x, w, None, False, 1e-6, r, dy)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("cols", [60, 3000, 30000])
def test_without_parameters(cols, layer):
    x, dy = inputs(6, cols, BF, 1).cuda(), inputs(6, cols, BF, 2).cuda()
    run(x, None, None, layer, 1e-5, dy=dy)
    _, b = (t.cuda() for t in params(cols, F))
    if layer:
        y = la.layer_norm(x, None, b)[0]
        y64, m, r = forward64(x.cpu(), None, b.cpu(), 1e-5, True)
        within(y, y64, forward_bound(x.cpu(), None, b.cpu(), 1e-5, True, y64, m, r, BF)[0], "y")


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("heads,cols,wide", [(5, 128, 9 * 128), (3, 33, 120), (2, 1030, 2061)])
def test_heads_inside_wider_rows(heads, cols, wide, dtype):
    """Rows with two strides, an odd start; what lies around outputs is left."""
    tokens = 70
    buffer = inputs(tokens, wide + 1, dtype, 1).cuda()
    x = buffer[:, 1:1 + heads * cols].unflatten(1, (heads, cols))
    dy = inputs(tokens * heads, cols, dtype, 2).cuda().reshape(tokens, heads, cols)
    w, b = (t.cuda() for t in params(cols, dtype))
    outs = [torch.full((tokens, wide + 1), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    inside = [o[:, 1:1 + heads * cols].unflatten(1, (heads, cols)) for o in outs]
    got = run(x, w, b, True, 1e-5, dy=dy, out=inside[0])
    back = la.layer_norm_backward(dy, x, w, got[1], dx=inside[1])
    assert torch.equal(back[0], got[2]) and back[0] is inside[1]
    for o in outs:
        assert bool((o[:, 0] == 7).all()) and bool((o[:, 1 + heads * cols:] == 7).all())


def test_heads_first_and_more_axes():
    x = inputs(2 * 3 * 4, 40, BF, 1).cuda().reshape(2, 3, 4, 40)
    w, b = (t.cuda() for t in params(40, BF))
    run(x.transpose(1, 2).contiguous().transpose(1, 2)[0], w, b, True, 1e-5,
        dy=inputs(12, 40, BF, 2).cuda().reshape(3, 4, 40))
    run(x, w, b, True, 1e-5, dy=x)
    run(x[0, 0, 0], w, b, True, 1e-5, dy=x[1, 1, 1])


def test_broadcast_inputs():
    """Inputs whose rows are one row: read only, so they may."""
    x = inputs(6, 100, BF, 1).cuda()
    r = inputs(1, 100, BF, 2).cuda().expand(6, 100)
    dy = inputs(1, 100, BF, 3).cuda().expand(6, 100)
    w, b = (t.cuda() for t in params(100, BF))
    run(x, w, b, True, 1e-5, r, dy, r)


@pytest.mark.parametrize("cols", [50, 5000, 40000])
def test_not_finite_rows_stay_apart(cols):
    x, dy = inputs(7, cols, BF, 1).cuda(), inputs(7, cols, BF, 2).cuda()
    w, b = (t.cuda() for t in params(cols, BF))
    y0, stats0 = la.layer_norm(x, w, b)
    dx0 = la.layer_norm_backward(dy, x, w, stats0)[0]
    x[2, 3], x[5, cols - 1] = float("nan"), float("inf")
    y, stats = la.layer_norm(x, w, b)
    dx, dw, db = la.layer_norm_backward(dy, x, w, stats)
    keep = torch.tensor([0, 1, 3, 4, 6])
    assert torch.equal(y[keep], y0[keep]) and torch.equal(dx[keep], dx0[keep])
    assert bool(y[[2, 5]].isnan().any(1).all()) and bool(dx[[2, 5]].isnan().any(1).all())
    assert bool(dw[3].isnan()) and bool(db.isfinite().all())


def test_zero_rows_and_zero_eps():
    x = torch.zeros(3, 70, device="cuda")
    w, b = (t.cuda() for t in params(70, F))
    y, stats = la.layer_norm(x, w, b, eps=1e-5)
    assert torch.equal(y, b.expand(3, 70)) and bool((stats[0] == 0).all())
    assert bool(la.rms_norm(x, w, eps=0.0)[0].isnan().all())
    run(inputs(3, 70, F, 1).cuda(), w, b, True, 0.0, dy=inputs(3, 70, F, 2).cuda())


def test_no_rows():
    x = torch.empty(0, 70, dtype=BF, device="cuda")
    w, b = (t.cuda() for t in params(70, BF))
    y, stats = la.layer_norm(x, w, b)
    assert y.shape == (0, 70) and stats.shape == (2, 0)
    dx, dw, db = la.layer_norm_backward(x, x, w, stats, dweight=torch.ones_like(w),
                                        dbias=torch.ones_like(b))
    assert dx.shape == (0, 70) and bool((dw == 0).all()) and bool((db == 0).all())
    y, stats = la.rms_norm(torch.empty(3, 0, device="cuda"))
    assert y.shape == (3, 0)


def test_what_is_not_wanted():
    x, dy = inputs(40, 300, BF, 1).cuda(), inputs(40, 300, BF, 2).cuda()
    w, b = (t.cuda() for t in params(300, BF))
    stats = la.layer_norm(x, w, b)[1]
    full = la.layer_norm_backward(dy, x, w, stats)
    dx, dw, db = la.layer_norm_backward(dy, x, w, stats, weight_grad=False, bias_grad=False)
    assert dw is None and db is None and torch.equal(dx, full[0])
    dx, dw, db = la.layer_norm_backward(dy, x, w, stats, weight_grad=False)
    assert dw is None and torch.equal(db, full[2])
    g32 = torch.empty(300, device="cuda")
    dw = la.layer_norm_backward(dy, x, w, stats, dweight=g32, bias_grad=False)[1]
    assert dw is g32 and torch.equal(g32.to(BF), full[1])


def test_the_same_bits_again_and_on_another_stream():
    x, dy = inputs(3000, 640, BF, 1).cuda(), inputs(3000, 640, BF, 2).cuda()
    w, b = (t.cuda() for t in params(640, BF))
    first = la.layer_norm(x, w, b) + la.layer_norm_backward(dy, x, w, la.layer_norm(x, w, b)[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, stats = la.layer_norm(x, w, b, stream=s)
    again = (y, stats) + la.layer_norm_backward(dy, x, w, stats, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for p, q in zip(first, again):
        assert torch.equal(p, q)


def test_captured():
    x, dy = inputs(100, 1000, BF, 1).cuda(), inputs(100, 1000, BF, 2).cuda()
    w, b = (t.cuda() for t in params(1000, BF))
    ws = torch.empty(la.norm_backward_workspace_bytes(x.shape, BF), dtype=torch.uint8,
                     device="cuda")
    outs = dict(out=torch.empty_like(x), stats=torch.empty(2, 100, device="cuda"))
    grads = dict(dx=torch.empty_like(x), dweight=torch.empty_like(w), dbias=torch.empty_like(b))

    def step():
        la.layer_norm(x, w, b, **outs)
        la.layer_norm_backward(dy, x, w, outs["stats"], workspace=ws, **grads)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        x.copy_(inputs(100, 1000, BF, 10 + k))
        for t in (*outs.values(), *grads.values()):
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        y, stats = la.layer_norm(x, w, b)
        want = (y, stats) + la.layer_norm_backward(dy, x, w, stats)
        for p, q in zip((*outs.values(), *grads.values()), want):
            assert torch.equal(p, q), k


def test_offsets_past_32_bits():
    stride = (1 << 31) + 24
    buffer = torch.empty(2 * stride + 100, dtype=BF, device="cuda")
    x = buffer.as_strided((3, 100), (stride, 1))
    x.copy_(inputs(3, 100, BF, 1))
    w, b = (t.cuda() for t in params(100, BF))
    run(x, w, b, True, 1e-5, dy=x)


def test_gradients_are_replicas_of_a_step():
    """dweight and dbias go to the AdamW step as they lie."""
    x, dy = inputs(64, 512, BF, 1).cuda(), (0.01 * inputs(64, 512, BF, 2)).to(BF).cuda()
    w, b = (t.cuda() for t in params(512, BF))
    _, dw, db = la.layer_norm_backward(dy, x, w, la.layer_norm(x, w, b)[1])
    state = [(t.float(), torch.zeros(512, device="cuda"), torch.zeros(512, device="cuda"), t.clone())
             for t in (w, b)]
    before = [s[0].clone() for s in state]
    la.step(state, [[dw], [db]], lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)
    for s, p, g in zip(state, before, (dw, db)):
        # the first step from zero moments is lr in the gradient's direction
        moved = (s[0] - p).double()
        g = g.double()
        want = -1e-3 * g / (g.abs() + 1e-8)
        assert float((moved - want).abs().max()) <= 1e-3 * 2.0 ** -20 + float(p.abs().max()) * 2.0 ** -23
