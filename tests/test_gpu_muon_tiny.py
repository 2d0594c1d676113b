"""Matrices with a short side of up to 16: strides, turned axes, in place,
empty and non-finite matrices, magnitudes, other polynomials, graphs, capped
grids, the flags of a step. Outputs in FP16 are within half a step of the
direction in 64 bits, and the directions themselves within 1.1e-5 (the
coefficients' rounding to 32 bits), which is added."""
import os
import subprocess
import sys

import pytest
import torch

import optimizer_step_layeradam_amd as la
import test_gpu_muon as steps
from muonhelpers import HALF_STEP, direction64, matrices, off

pytestmark = pytest.mark.gpu

BAR = HALF_STEP[torch.float16] + 1.1e-5
# one workgroup a matrix, and matrices cut into parts
SHAPES = [(7, 200), (16, 16), (3, 11, 90), (3000, 5), (2, 16, 1100), (1, 700), (2, 2, 513)]


def direction(x, **kw):
    # an empty() like x's layout, in FP16
    o = torch.empty_like(x, dtype=torch.float16)
    la.orthogonalize(x, o, **kw)
    return o


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_types(shape, dtype):
    x = matrices(shape, "spiked", seed=sum(shape), scale=1e-2).to(dtype).cuda()
    assert off(direction(x), direction64(x.cpu())) <= BAR
    b = la.orthogonalize(x, torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
    assert off(b, direction64(x.cpu())) <= HALF_STEP[torch.bfloat16] + 1.1e-5


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_strides_rows_apart_and_turned_axes(shape):
    full = matrices((*shape[:-2], 2 * shape[-2], shape[-1] + 13), seed=8).cuda()
    x = full[..., ::2, 5:5 + shape[-1]]
    guard = torch.full((*shape[:-2], 3 * shape[-2], shape[-1] + 7), 7.0, dtype=torch.float16,
                       device="cuda")
    o = guard[..., ::3, 3:3 + shape[-1]]
    la.orthogonalize(x, o)
    assert off(o, direction64(x.cpu())) <= BAR
    o.fill_(7.0)
    assert torch.all(guard == 7.0)  # nothing outside the view was written
    turned = torch.empty(shape, dtype=torch.float16, device="cuda")
    la.orthogonalize(x.mT, turned.mT)
    assert off(turned, direction64(x.cpu())) <= BAR


@pytest.mark.parametrize("rows", [16, 700])
def test_heads_side_by_side(rows):
    w = matrices((rows, 6 * 12), seed=9).to(torch.float16).cuda()  # 6 heads of 12 columns
    heads, o = w.view(rows, 6, 12).transpose(0, 1), torch.empty_like(w)
    la.orthogonalize(heads, o.view(rows, 6, 12).transpose(0, 1))
    assert off(o.view(rows, 6, 12).transpose(0, 1), direction64(heads.cpu())) <= BAR


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_in_place(shape):
    x = matrices(shape, seed=10).to(torch.float16).cuda()
    want = la.orthogonalize(x)
    y = x.clone()
    la.orthogonalize(y, y)
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("shape", [(5, 6, 70), (5, 900, 9)])
def test_zeros_stay_zero_and_nonfinite_matrices_are_nan_alone(shape):
    x = matrices(shape, seed=7)
    x[1] = 0.0
    x[2, -1, -1] = float("nan")
    x[3, 0, 0] = float("-inf")
    for eps in (1e-7, 0.0):
        o = la.orthogonalize(x.cuda(), torch.empty(shape, dtype=torch.float16, device="cuda"),
                             eps=eps).cpu()
        assert torch.all(o[1] == 0.0)
        assert torch.isnan(o[2]).all() and torch.isnan(o[3]).all()
        for z in (0, 4):
            assert off(o[z], direction64(x[z])) <= BAR


@pytest.mark.parametrize("shape", [(9, 200), (1500, 3)])
def test_magnitudes_do_not_matter_and_eps_bounds_the_norm(shape):
    x = matrices(shape, seed=5)
    ref = la.orthogonalize(x.cuda(), eps=0.0).cpu()
    for k in (-120, -60, 60, 110):
        y = la.orthogonalize((x * 2.0 ** k).cuda(), eps=0.0)
        assert torch.equal(y.cpu().view(torch.int16), ref.view(torch.int16)), k
    x = 1e-3 * x
    assert off(direction(x.cuda(), eps=1.0), direction64(x, eps=1.0)) <= BAR


@pytest.mark.parametrize("count", [1, 2, 6])
def test_other_polynomials(count):
    """Coefficients that 32 bits hold."""
    cubic = ((1.5, -0.5, 0.0),) * count
    mixed = (((2.0, -1.5, 0.5), (1.5, -0.5, 0.0)) * count)[:count]
    for shape in ((5, 80), (2000, 12)):
        x = matrices(shape, seed=11).cuda()
        for c in (cubic, mixed):
            assert off(direction(x, coefficients=c), direction64(x.cpu(), c)) <= BAR


def test_same_bits_on_any_workspace_and_nothing_written_behind_it():
    for shape in ((3, 9, 40), (2, 7, 3000)):
        x = matrices(shape, seed=13).to(torch.bfloat16).cuda()
        first = la.orthogonalize(x)
        need = la.orthogonalize_workspace_bytes([shape])
        for fill in (0, 0xFF):
            ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
            again = la.orthogonalize(x, workspace=ws[:need])
            assert torch.equal(first.view(torch.int16), again.view(torch.int16))
            assert torch.all(ws[need:] == fill)


def test_captured_and_replayed():
    x = [matrices(s, seed=18).to(torch.bfloat16).cuda() for s in ((2, 15, 310), (8, 4000))]
    o = [torch.empty_like(t) for t in x]
    la.orthogonalize(x, o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        la.orthogonalize(x, o)
    for k in range(4):
        for t in x:
            t.copy_(matrices(t.shape, seed=20 + k))
        want = la.orthogonalize(x)
        for t in o:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for t, w in zip(o, want):
            assert torch.equal(t.view(torch.int16), w.view(torch.int16)), k


STEP_SHAPES = [(1, 1), (16, 16), (3, 5, 9), (2, 3000, 7), (1, 900), (20, 11, 30)]


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("R,dtype", [(1, torch.bfloat16), (3, torch.float16)])
def test_steps(R, dtype, nesterov):
    for out in (torch.bfloat16, torch.float16, None):
        params, grads = steps.make(STEP_SHAPES, R, dtype, out, seed=50 + R)
        hyper = dict(lr=1e-2, weight_decay=0.1, nesterov=nesterov, grad_unscale=0.5)
        ref = steps.reference(params, grads, **hyper)
        la.muon_step(params, grads, **hyper)
        steps.check(params, ref)


def test_flag_and_skip():
    params, grads = steps.make(STEP_SHAPES, 1, torch.bfloat16, torch.bfloat16, seed=70)
    skip = torch.ones(1, dtype=torch.int32, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = [[t.clone() for t in x] for x in params]
    grads[3][0][1, 2999, 6] = float("inf")
    la.muon_step(params, grads, lr=1e-2, overflow_flag=flag, skip_if_nonzero=skip)
    assert int(flag) == 0
    assert all(torch.equal(a, b) for x, y in zip(params, before) for a, b in zip(x, y))
    skip.zero_()
    ref = steps.reference(params, grads, lr=1e-2)
    la.muon_step(params, grads, lr=1e-2, overflow_flag=flag, skip_if_nonzero=skip)
    assert int(flag) == 1
    assert torch.isnan(params[3][0][1]).all() and not torch.isnan(params[3][0][0]).any()
    steps.check([x for i, x in enumerate(params) if i != 3], [r for i, r in enumerate(ref) if i != 3])


def test_more_stacks_than_one_launch_takes():
    xs = [matrices((1 + i % 3, 1 + 7 * i % 16, 1 + 131 * i % 1500), seed=i).cuda()
          for i in range(40)]
    outs = [torch.empty_like(x, dtype=torch.float16) for x in xs]
    la.orthogonalize(xs, outs)
    for x, o in zip(xs, outs):
        assert off(o, direction64(x.cpu())) <= BAR


@pytest.mark.parametrize("cap", [1, 5])
def test_striding_loops_under_a_capped_grid(cap):
    child = os.path.join(os.path.dirname(__file__), "muon_tiny_child.py")
    env = dict(os.environ, LAYERADAM_MAX_GRID=str(cap))
    r = subprocess.run([sys.executable, child], env=env, capture_output=True, text=True,
                       timeout=100)
    print(r.stdout[-2000:], flush=True)
    assert r.returncode == 0, r.stderr[-2000:]
