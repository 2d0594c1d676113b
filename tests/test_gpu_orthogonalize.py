"""The orthogonalised update on the GPU against its polynomial in 64 bits."""
import os
import subprocess
import sys

import pytest
import torch

import optimizer_step_layeradam_amd as la
from muonhelpers import DIRECTION, HALF_STEP, direction64, matrices, off

pytestmark = pytest.mark.gpu

# Sides on both sides of the tiles (64, 128, 256) and of the padding, single
# rows and columns, wide and tall, stacks whose matrices start unaligned.
SHAPES = [(1, 1), (1, 7), (9, 1), (1, 1000), (5, 3), (31, 33), (63, 65), (64, 64), (65, 63),
          (100, 260), (127, 129), (128, 128), (129, 127), (255, 257), (256, 256), (257, 255),
          (300, 1100), (1100, 300), (513, 515), (3, 5, 9), (4, 64, 64), (7, 33, 70),
          (2, 130, 100), (5, 17, 1030), (3, 1000, 24), (2, 300, 300)]


def check(x, out, **kw):
    ref = direction64(x.cpu(), **kw)
    tol = DIRECTION + HALF_STEP[out.dtype]
    got = off(out, ref)
    print(f"  {tuple(x.shape)} {x.dtype} -> {out.dtype}: off {got:.2e} (bar {tol:.2e})",
          flush=True)
    assert out.shape == x.shape
    assert got <= tol


@pytest.mark.parametrize("kind", ["gauss", "lowrank", "spiked", "outliers"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes_and_spectra(shape, kind):
    x = matrices(shape, kind, seed=len(shape) + shape[-1]).cuda()
    check(x, la.orthogonalize(x))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_types(dtype, out):
    for shape in ((2, 77, 131), (150, 90)):
        x = matrices(shape, seed=3, scale=1e-2).to(dtype).cuda()
        o = torch.empty(shape, dtype=out, device="cuda")
        assert la.orthogonalize(x, o) is o
        check(x, o)


@pytest.mark.parametrize("least", [1, 129])
def test_many_stacks_in_one_call_equal_one_call_each(least):
    """37 stacks, narrow ones (short side up to 128) or wide ones, take the same
    form together as alone, and so give the same bits."""
    xs = [matrices((1 + i % 3, least + 13 * i % 120, least + 29 * i % 127), seed=i)
          .to(torch.bfloat16).cuda() for i in range(37)]
    together = la.orthogonalize(xs)
    for x, o in zip(xs, together):
        alone = la.orthogonalize(x)
        assert torch.equal(o.view(torch.int16), alone.view(torch.int16)), x.shape


def test_narrow_and_wide_stacks_in_one_call():
    shapes = [(1 + i % 3, 1 + 13 * i % 150, 1 + 29 * i % 170) for i in range(37)]
    shapes += [(40, 100, 1100), (20, 4200, 60)]  # narrow ones of their own launches
    xs = [matrices(s, seed=i).to(torch.bfloat16).cuda() for i, s in enumerate(shapes)]
    for x, o in zip(xs, la.orthogonalize(xs)):
        check(x, o)


@pytest.mark.parametrize("shape", [(128, 5000), (5000, 127), (64, 3001), (2999, 65), (1, 12000),
                                   (12000, 2), (3, 33, 2000), (5, 1500, 100), (600, 20, 50),
                                   (513, 70, 90), (128, 513), (64, 512), (514, 128)], ids=str)
@pytest.mark.parametrize("kind", ["gauss", "lowrank", "spiked"])
def test_long_narrow_matrices_and_many_of_them(shape, kind):
    x = matrices(shape, kind, seed=sum(shape)).cuda()
    check(x, la.orthogonalize(x))


def test_magnitudes_do_not_matter():
    x = matrices((96, 200), seed=5)
    ref = la.orthogonalize(x.cuda()).cpu()
    for k in (-100, -60, 60, 100):  # the squares of these leave binary32
        y = la.orthogonalize((x * 2.0 ** k).cuda(), eps=0.0)
        assert torch.equal(y.cpu().view(torch.int16), ref.view(torch.int16)), k


def test_eps_bounds_the_norm_from_below():
    x = matrices((40, 90), seed=6, scale=1e-3)
    check(x.cuda(), la.orthogonalize(x.cuda(), eps=1.0), eps=1.0)


def test_zeros_stay_zero_and_nonfinite_matrices_are_nan_alone():
    x = matrices((5, 70, 150), seed=7)
    x[1] = 0.0
    x[2, 69, 149] = float("nan")
    x[3, 0, 0] = float("-inf")
    for eps in (1e-7, 0.0):
        o = la.orthogonalize(x.cuda(), eps=eps).cpu()
        assert torch.all(o[1] == 0.0)
        assert torch.isnan(o[2]).all() and torch.isnan(o[3]).all()
        for z in (0, 4):
            assert off(o[z], direction64(x[z])) <= DIRECTION + HALF_STEP[torch.bfloat16]


@pytest.mark.parametrize("shape", [(60, 100), (3, 60, 100), (200, 90)])
def test_strides_rows_apart_and_turned_axes(shape):
    full = matrices((*shape[:-2], 2 * shape[-2], shape[-1] + 13), seed=8).cuda()
    x = full[..., ::2, 5:5 + shape[-1]]
    guard = torch.full((*shape[:-2], 3 * shape[-2], shape[-1] + 7), 7.0, dtype=torch.bfloat16,
                       device="cuda")
    o = guard[..., ::3, 3:3 + shape[-1]]
    la.orthogonalize(x, o)
    check(x, o)
    o.fill_(7.0)
    assert torch.all(guard == 7.0)  # nothing outside the view was written
    turned = x.mT
    out = la.orthogonalize(turned)
    assert out.stride(-2) == 1
    check(turned, out)


def test_heads_side_by_side():
    w = matrices((96, 5 * 48), seed=9).to(torch.bfloat16).cuda()  # 5 heads of 48 columns
    heads = w.view(96, 5, 48).transpose(0, 1)
    o = torch.empty_like(w)
    la.orthogonalize(heads, o.view(96, 5, 48).transpose(0, 1))
    check(heads, o.view(96, 5, 48).transpose(0, 1))


@pytest.mark.parametrize("shape", [(2, 50, 300), (140, 33)])
def test_in_place(shape):
    x = matrices(shape, seed=10).to(torch.float16).cuda()
    want = la.orthogonalize(x)
    y = x.clone()
    la.orthogonalize(y, y)
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("steps", [1, 2, 3, 10])
def test_other_polynomials(steps):
    # the cubic 3/2, -1/2: converges for every singular value in (0, sqrt 3)
    cubic = ((1.5, -0.5, 0.0),) * steps
    x = matrices((48, 130), seed=11).cuda()
    check(x, la.orthogonalize(x, coefficients=cubic), coefficients=cubic)
    mixed = (((4.0, -6.0, 2.5), (2.0, -1.5, 0.5)) * steps)[:steps]
    check(x, la.orthogonalize(x, coefficients=mixed), coefficients=mixed)


def test_ten_cubic_steps_give_orthogonal_rows():
    q = torch.linalg.qr(matrices((60, 60), seed=12).double())[0]
    x = (q * torch.linspace(0.5, 1.5, 60).double()).float().cuda()
    o = la.orthogonalize(x, coefficients=((1.5, -0.5, 0.0),) * 10).double().cpu()
    # ||X_0|| = 1: singular values start at 0.06 .. 0.19 and end at 1; each
    # entry of O O^T sums 60 products of entries a half step of BF16 off
    assert (o @ o.mT - torch.eye(60, dtype=torch.float64)).abs().max() < 2 * 2.0 ** -8 + 4 * DIRECTION


def test_same_bits_every_time_and_on_any_workspace():
    x = matrices((3, 200, 333), seed=13).to(torch.bfloat16).cuda()
    first = la.orthogonalize(x)
    need = la.orthogonalize_workspace_bytes([tuple(x.shape)])
    for fill in (0, 0xFF, 0x7C):  # what the workspace holds before the call means nothing
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        again = la.orthogonalize(x, workspace=ws)
        assert torch.equal(first.view(torch.int16), again.view(torch.int16)), fill


def test_nothing_behind_the_workspace_is_written():
    for shape in ((1, 1), (3, 65, 130), (129, 257)):
        need = la.orthogonalize_workspace_bytes([shape])
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        la.orthogonalize(matrices(shape, seed=14).cuda(), workspace=ws[:need])
        assert torch.all(ws[need:] == 0xA5)


def test_empty_stacks_are_skipped():
    x = [torch.empty(s, device="cuda") for s in ((0, 5), (5, 0), (0, 3, 3))]
    y = matrices((20, 30), seed=15).cuda()
    out = la.orthogonalize([*x, y])
    check(y, out[-1])
    assert la.orthogonalize([]) == []


def test_another_stream_and_two_at_once():
    a, b = matrices((400, 700), seed=16).cuda(), matrices((2, 300, 500), seed=17).cuda()
    want = la.orthogonalize(a), la.orthogonalize(b)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        x, y = la.orthogonalize(a, stream=s), la.orthogonalize(b, stream=t)
        torch.cuda.synchronize()
        assert torch.equal(x.view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(y.view(torch.int16), want[1].view(torch.int16))


def test_captured_and_replayed():
    x = matrices((2, 150, 310), seed=18).to(torch.bfloat16).cuda()
    o = torch.empty_like(x)
    la.orthogonalize(x, o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        la.orthogonalize(x, o)
    for k in range(4):
        x.copy_(matrices(x.shape, seed=20 + k))
        want = la.orthogonalize(x)
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.view(torch.int16), want.view(torch.int16)), k


@pytest.mark.parametrize("cap", [1, 7])
def test_striding_loops_under_a_capped_grid(cap):
    child = os.path.join(os.path.dirname(__file__), "muon_stride_child.py")
    env = dict(os.environ, LAYERADAM_MAX_GRID=str(cap))
    r = subprocess.run([sys.executable, child], env=env, capture_output=True, text=True,
                       timeout=100)
    print(r.stdout[-2000:], flush=True)
    assert r.returncode == 0, r.stderr[-2000:]
