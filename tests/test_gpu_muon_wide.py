"""The step-by-step form of the orthogonalised update (short sides past 128,
or a polynomial that the narrow form is not precise enough for): the same
properties as the narrow form's, on sides that take it. And what both share
where workspaces meet graphs and streams."""
import pytest
import torch

import optimizer_step_layeradam_amd as la
import test_gpu_muon as steps
from muonhelpers import DIRECTION, HALF_STEP, QUINTIC, direction64, matrices, off
from test_gpu_orthogonalize import check

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view(torch.int16)


# Enough tiles that 256 x 256 ones are the fewest rounds: odd sides, wide and tall.
LARGE = [(25, 513, 515), (26, 700, 516)]


@pytest.mark.parametrize("kind", ["gauss", "lowrank"])
@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_largest_tiles(shape, kind):
    x = matrices(shape, kind, seed=200).cuda()
    check(x, la.orthogonalize(x))


@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_largest_tiles_in_a_step(shape):
    params, grads = steps.make([shape], 2, torch.float16, torch.bfloat16, seed=201)
    ref = steps.reference(params, grads, lr=1e-2, weight_decay=0.1)
    la.muon_step(params, grads, lr=1e-2, weight_decay=0.1)
    steps.check(params, ref)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_types(dtype, out):
    for shape in ((2, 140, 333), (260, 150), (136, 264)):
        x = matrices(shape, seed=202, scale=1e-2).to(dtype).cuda()
        o = torch.empty(shape, dtype=out, device="cuda")
        la.orthogonalize(x, o)
        check(x, o)


@pytest.mark.parametrize("shape", [(150, 200), (2, 150, 200), (300, 140)])
def test_strides_rows_apart_and_turned_axes(shape):
    full = matrices((*shape[:-2], 2 * shape[-2], shape[-1] + 13), seed=203).cuda()
    x = full[..., ::2, 5:5 + shape[-1]]
    guard = torch.full((*shape[:-2], 3 * shape[-2], shape[-1] + 7), 7.0, dtype=torch.bfloat16,
                       device="cuda")
    o = guard[..., ::3, 3:3 + shape[-1]]
    la.orthogonalize(x, o)
    check(x, o)
    o.fill_(7.0)
    assert torch.all(guard == 7.0)
    turned = x.mT
    out = la.orthogonalize(turned)
    assert out.stride(-2) == 1
    check(turned, out)


@pytest.mark.parametrize("cols", [160, 141])
def test_heads_side_by_side(cols):
    w = matrices((144, 3 * cols), seed=204).to(torch.bfloat16).cuda()
    heads = w.view(144, 3, cols).transpose(0, 1)
    o = torch.empty_like(w)
    la.orthogonalize(heads, o.view(144, 3, cols).transpose(0, 1))
    check(heads, o.view(144, 3, cols).transpose(0, 1))


@pytest.mark.parametrize("shape", [(2, 200, 333), (340, 133)])
def test_in_place(shape):
    x = matrices(shape, seed=205).to(torch.float16).cuda()
    want = la.orthogonalize(x)
    y = x.clone()
    la.orthogonalize(y, y)
    assert torch.equal(bits(y), bits(want))


def test_magnitudes_do_not_matter():
    x = matrices((150, 210), seed=206)
    ref = la.orthogonalize(x.cuda()).cpu()
    for k in (-100, -60, 60, 100):
        y = la.orthogonalize((x * 2.0 ** k).cuda(), eps=0.0)
        assert torch.equal(bits(y.cpu()), bits(ref)), k


def test_eps_bounds_the_norm_from_below():
    x = matrices((140, 190), seed=207, scale=1e-3)
    check(x.cuda(), la.orthogonalize(x.cuda(), eps=2.0), eps=2.0)


def test_zeros_stay_zero_and_nonfinite_matrices_are_nan_alone():
    x = matrices((5, 140, 300), seed=208)
    x[1] = 0.0
    x[2, 139, 299] = float("nan")
    x[3, 0, 0] = float("-inf")
    for eps in (1e-7, 0.0):
        o = la.orthogonalize(x.cuda(), eps=eps).cpu()
        assert torch.all(o[1] == 0.0)
        assert torch.isnan(o[2]).all() and torch.isnan(o[3]).all()
        for z in (0, 4):
            assert off(o[z], direction64(x[z])) <= DIRECTION + HALF_STEP[torch.bfloat16]


@pytest.mark.parametrize("count", [1, 2, 3, 10])
def test_other_polynomials(count):
    cubic = ((1.5, -0.5, 0.0),) * count
    for shape in ((150, 260), (270, 140)):
        x = matrices(shape, seed=209).cuda()
        check(x, la.orthogonalize(x, coefficients=cubic), coefficients=cubic)
        mixed = (((4.0, -6.0, 2.5), (2.0, -1.5, 0.5)) * count)[:count]
        check(x, la.orthogonalize(x, coefficients=mixed), coefficients=mixed)


@pytest.mark.parametrize("count", [1, 2])
def test_few_steps_of_a_muon_step(count):
    """One and two steps: the direction's place in the workspace is larger than
    the second iterate that it shares it with."""
    params, grads = steps.make([(150, 260), (300, 133)], 1, torch.bfloat16, None, seed=210)
    cubic = ((1.5, -0.5, 0.0),) * count
    us = [g[0].float() + 0.95 * (0.95 * p[1] + g[0].float()) for p, g in zip(params, grads)]
    for p in params:
        p[0].zero_()
    la.muon_step(params, grads, lr=1.0, lr_scale="none", coefficients=cubic)
    for p, u in zip(params, us):
        assert off(-p[0], direction64(u.cpu(), cubic)) <= DIRECTION


@pytest.mark.parametrize("shape", [(48, 130), (20, 500), (1, 9), (9, 1), (600, 20, 50),
                                   (3, 900, 70), (64, 64)], ids=str)
def test_narrow_matrices_under_a_polynomial_of_large_growth(shape):
    """Six steps: the factor reaches past 512, and so the step-by-step form is
    taken. Each step has the part of the bar that it has among five."""
    six = QUINTIC + QUINTIC[:1]
    for kind in ("gauss", "lowrank"):
        x = matrices(shape, kind, seed=211).cuda()
        got = off(la.orthogonalize(x, coefficients=six), direction64(x.cpu(), six))
        print(f"  {shape} {kind}: {got:.2e}", flush=True)
        assert got <= 6 / 5 * DIRECTION + HALF_STEP[torch.bfloat16]


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [(40, 100, 1100), (128, 5000), (3000, 70), (520, 30, 600),
                                   (514, 64, 64), (513, 700, 9), (2, 65, 2049)], ids=str)
def test_long_narrow_matrices_and_many_of_them_in_a_step(shape, nesterov):
    params, grads = steps.make([shape], 1, torch.bfloat16, torch.bfloat16, seed=212)
    hp = dict(lr=1e-2, weight_decay=0.1, nesterov=nesterov)
    ref = steps.reference(params, grads, **hp)
    la.muon_step(params, grads, **hp)
    steps.check(params, ref)


def test_flag_and_nan_stay_with_their_matrix():
    params, grads = steps.make([(3, 140, 150), (233, 200)], 2, torch.float16, torch.float16,
                               seed=213)
    grads[0][1][1, 139, 149] = float("inf")
    ref = steps.reference(params, grads, lr=1e-2)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    la.muon_step(params, grads, lr=1e-2, overflow_flag=flag)
    assert flag.item() == 1
    p, m, _ = params[0]
    assert torch.isnan(p[1]).all() and torch.isinf(m[1, 139, 149])
    steps.check([tuple(x[::2] for x in params[0]), params[1]],
                [tuple(x[::2] for x in ref[0]), ref[1]])


def test_skip_leaves_everything_as_it_was():
    params, grads = steps.make([(170, 190), (2, 140, 300), (2, 20, 3000)], 2, torch.bfloat16,
                               torch.bfloat16, seed=214)
    keep = [[t.clone() for t in x] for x in params]
    layer = la.MuonLayer(params, grads,
                         torch.full((1 << 24,), 0xA5, dtype=torch.uint8, device="cuda"))
    assert layer.workspace_bytes() <= 1 << 24
    skip = torch.ones(1, dtype=torch.int32, device="cuda")
    layer.step(lr=1e-2, skip_if_nonzero=skip)
    for x, y in zip(params, keep):
        for a, b in zip(x, y):
            assert torch.equal(a, b)
    assert torch.all(layer._workspace == 0xA5)
    skip.zero_()
    ref = steps.reference(params, grads, lr=1e-2)
    layer.step(lr=1e-2, skip_if_nonzero=skip)
    steps.check(params, ref)


def test_nothing_behind_the_workspace_is_written():
    shapes = [(150, 260), (3, 300, 133), (129, 129)]
    for coefficients in (None, ((1.5, -0.5, 0.0),), ((1.5, -0.5, 0.0),) * 2):
        params, grads = steps.make(shapes, 1, torch.bfloat16, None, seed=215)
        need = la.MuonLayer(params, grads).workspace_bytes(coefficients=coefficients)
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        la.muon_step(params, grads, lr=1e-2, coefficients=coefficients, workspace=ws[:need])
        assert torch.all(ws[need:] == 0xA5)


def test_pinned_host_state():
    params, grads = steps.make([(150, 260)], 1, torch.bfloat16, None, seed=216)
    ref = steps.reference(params, grads, lr=1e-2)
    host = [tuple(torch.empty(t.shape, pin_memory=True).copy_(t) for t in params[0][:2])]
    la.muon_step(host, grads, lr=1e-2)
    torch.cuda.synchronize()
    steps.check(host, ref)


def test_two_steps_at_once_on_two_streams():
    sets = [steps.make(s, 1, torch.bfloat16, torch.bfloat16, seed=217 + i)
            for i, s in enumerate(([(400, 700), (60, 900)], [(2, 300, 500), (70, 70)]))]
    refs = [steps.reference(*x, lr=1e-2) for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for x, s in zip(sets, streams):
        la.muon_step(*x, lr=1e-2, stream=s)
    torch.cuda.synchronize()
    for x, ref in zip(sets, refs):
        steps.check(x[0], ref)


def test_two_graphs_share_a_workspace_in_turn():
    sets = [steps.make(s, 1, torch.bfloat16, torch.bfloat16, seed=220 + i)
            for i, s in enumerate(([(200, 300), (60, 900)], [(3, 150, 140), (10, 10)]))]
    layers = [la.MuonLayer(*x) for x in sets]
    ws = torch.empty(max(x.workspace_bytes() for x in layers), dtype=torch.uint8, device="cuda")
    layers = [la.MuonLayer(*x, workspace=ws) for x in sets]
    graphs = []
    for layer in layers:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            layer.step(lr=1e-2)
    for _ in range(3):
        refs = [steps.reference(*x, lr=1e-2) for x in sets]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, ref in zip(sets, refs):
            steps.check(x[0], ref)


def test_step_captured_by_itself():
    """muon_step with its workspace from the capture's own pool, between other
    allocations there."""
    params, grads = steps.make([(200, 300), (5, 40, 60)], 1, torch.bfloat16, None, seed=230)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.muon_step(params, grads, lr=1e-2)
        after = torch.zeros(1 << 20, device="cuda")
        after.add_(params[0][1].sum())
    for _ in range(3):
        ref = steps.reference(params, grads, lr=1e-2)
        graph.replay()
        torch.cuda.synchronize()
        steps.check(params, ref)


def test_a_captured_step_keeps_its_workspace():
    """A later step that needs more takes a new workspace; the old one stays
    the graph's."""
    params, grads = steps.make([(150, 260)], 1, torch.bfloat16, None, seed=240)
    layer = la.MuonLayer(params, grads)
    small = dict(lr=1e-2, nesterov=False, coefficients=((1.5, -0.5, 0.0),))
    layer.step(**small)
    size, place = layer._workspace.numel(), layer._workspace.data_ptr()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(**small)
    layer.step(lr=1e-2)
    assert layer._workspace.numel() > size
    others = [torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(t.data_ptr() != place for t in others)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.all(t == 0xA5) for t in others)
