"""The norms on the host: argument checks of the C ABI and of the binding,
workspace sizes, and the formulas that the GPU tests compare with against
differentiation and against differences. No kernel runs here.

The calls with made-up device addresses are all invalid on purpose and must be
refused on the host; they are skipped where a GPU is visible, so that no such
address can reach a device.
"""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import optimizer_step_layeradam_amd as la
from normhelpers import backward64, forward64, inputs, params

host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="uses made-up device addresses; host-only check")

BASE = 0x7F0000000000
STEP = 0x1000000000
WS = BASE + 0x100 * STEP
OK, INVALID, MISALIGNED, ALIASING, UNSUPPORTED = 0, 1, 2, 3, 4
OUTER, INNER, COLS = 5, 3, 40


def at(k, offset=0):
    return BASE + k * STEP + offset


def rows(k, outer=INNER * COLS, inner=COLS, offset=0):
    return la.Rows(at(k, offset) if k is not None else 0, outer, inner)


def norm(**kw):
    a = dict(kind=la.NORM_LAYER, outer=OUTER, inner=INNER, cols=COLS, type=la.TYPE_BF16,
             weight_type=la.TYPE_FP32, weight=at(10), bias=at(11), eps=1e-5)
    return la.make_norm(**dict(a, **kw))


NONE = la.Rows(0, 0, 0)


def forward_io(**kw):
    a = dict(x=rows(0), residual=rows(1), y=rows(2), sum=rows(3), mean=at(4), rstd=at(5))
    a.update(kw)
    return la.NormForwardIO(a["x"], a["residual"], a["y"], a["sum"], a["mean"], a["rstd"])


def backward_io(**kw):
    a = dict(dy=rows(0), x=rows(1), residual_grad=rows(2), dx=rows(3), mean=at(4), rstd=at(5),
             dweight=at(6), dbias=at(7), grad_type=la.TYPE_BF16)
    a.update(kw)
    return la.NormBackwardIO(*[a[f] for f, _ in la.NormBackwardIO._fields_])


def refuses(status, call):
    with pytest.raises(la.LayerAdamError) as e:
        call()
    assert e.value.status == status, str(e.value)
    assert la.last_error()


def test_structs_have_the_sizes_of_the_header():
    names = {"la_rows": la.Rows, "la_norm_desc": la.NormDesc,
             "la_norm_forward_io": la.NormForwardIO, "la_norm_backward_io": la.NormBackwardIO}
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with tempfile.TemporaryDirectory() as d:
        src = os.path.join(d, "t.c")
        with open(src, "w") as f:
            f.write('#include "layeradam.h"\n#include <stdio.h>\nint main(void){' + "".join(
                f'printf("%zu\\n", sizeof({n}));' for n in names) + "return 0;}\n")
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), src, "-o",
                        os.path.join(d, "t")], check=True)
        sizes = subprocess.run([os.path.join(d, "t")], capture_output=True, text=True,
                               check=True).stdout.split()
    assert [int(s) for s in sizes] == [ctypes.sizeof(c) for c in names.values()]


@host_only
@pytest.mark.parametrize("kw,status", [
    (dict(kind=2), UNSUPPORTED), (dict(type=3), UNSUPPORTED), (dict(weight_type=-1), UNSUPPORTED),
    (dict(outer=-1), INVALID), (dict(inner=-1), INVALID), (dict(cols=-1), INVALID),
    (dict(cols=la.MAX_SIDE + 1), INVALID), (dict(outer=1 << 32), INVALID),
    (dict(outer=1 << 30, inner=1 << 30), INVALID),
    (dict(eps=-1e-9), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(eps=1e39), INVALID),
    (dict(weight=at(10, 2)), MISALIGNED), (dict(bias=at(11, 1)), MISALIGNED),
    (dict(weight=at(2, 8)), ALIASING), (dict(bias=at(3, 8)), ALIASING),
])
def test_refuses_descriptors(kw, status):
    refuses(status, lambda: la.norm_forward_raw(norm(**kw), forward_io()))
    if "bias" not in kw and status != ALIASING:
        refuses(status, lambda: la.norm_backward_raw(norm(**kw), backward_io(), WS, 1 << 30))


LAST = 2 * (OUTER * INNER * COLS - 1)


@host_only
@pytest.mark.parametrize("kw,status", [
    (dict(x=rows(None)), INVALID), (dict(y=rows(None)), INVALID),
    (dict(residual=NONE), INVALID), (dict(sum=NONE), INVALID),
    (dict(x=rows(0, offset=1)), MISALIGNED), (dict(y=rows(2, offset=1)), MISALIGNED),
    (dict(mean=at(4, 2)), MISALIGNED), (dict(rstd=at(5, 1)), MISALIGNED),
    (dict(x=rows(0, outer=-120)), INVALID), (dict(x=rows(0, inner=1 << 41)), INVALID),
    (dict(y=rows(2, inner=39)), INVALID), (dict(y=rows(2, outer=119)), INVALID),
    (dict(y=rows(2, outer=0)), INVALID), (dict(sum=rows(3, inner=0)), INVALID),
    (dict(y=rows(2, outer=40, inner=199)), INVALID),
    (dict(y=rows(0)), ALIASING), (dict(y=rows(0, offset=LAST)), ALIASING),
    (dict(sum=rows(2, offset=LAST)), ALIASING), (dict(sum=rows(1)), ALIASING),
    (dict(mean=at(5, 4 * 14)), ALIASING), (dict(rstd=at(0)), ALIASING),
])
def test_refuses_forward(kw, status):
    refuses(status, lambda: la.norm_forward_raw(norm(), forward_io(**kw)))


@host_only
@pytest.mark.parametrize("kw,status", [
    (dict(dy=rows(None)), INVALID), (dict(x=rows(None)), INVALID), (dict(rstd=0), INVALID),
    (dict(mean=0), INVALID), (dict(grad_type=5), UNSUPPORTED),
    (dict(dy=rows(0, offset=1)), MISALIGNED), (dict(dx=rows(3, offset=1)), MISALIGNED),
    (dict(dweight=at(6, 1)), MISALIGNED), (dict(dbias=at(7, 2), grad_type=la.TYPE_FP32), MISALIGNED),
    (dict(residual_grad=rows(2, offset=1)), MISALIGNED),
    (dict(dx=rows(3, inner=20)), INVALID), (dict(dy=rows(0, inner=-1)), INVALID),
    (dict(dx=rows(0)), ALIASING), (dict(dx=rows(2, offset=LAST)), ALIASING),
    (dict(dweight=at(7, 2 * COLS - 2)), ALIASING), (dict(dweight=at(10)), ALIASING),
    (dict(dbias=WS + 64), ALIASING), (dict(x=la.Rows(WS, 0, 0)), ALIASING),
])
def test_refuses_backward(kw, status):
    refuses(status, lambda: la.norm_backward_raw(norm(), backward_io(**kw), WS, 1 << 30))


@host_only
def test_refuses_workspaces():
    need = la.norm_backward_workspace_bytes_raw(norm())
    assert need > 0
    for ws, size, status in ((0, need, INVALID), (WS + 128, need, MISALIGNED),
                             (WS, need - 1, INVALID), (WS, -1, INVALID), (at(3), need, ALIASING)):
        refuses(status, lambda: la.norm_backward_raw(norm(), backward_io(), ws, size))


@host_only
@pytest.mark.parametrize("outer,inner", [(1 << 30, 1), (1, 1 << 30), (1 << 20, 1 << 10)])
def test_refuses_tensors_past_any_address(outer, inner):
    # rows times stride would pass 64 bits, each alone is allowed
    far = (1 << 40) - 1
    n = norm(outer=outer, inner=inner, weight=0, bias=0, cols=8)
    for kw in (dict(x=la.Rows(at(0), far, far)), dict(y=la.Rows(at(2), far, far))):
        refuses(INVALID, lambda: la.norm_forward_raw(
            n, forward_io(residual=NONE, sum=NONE, mean=0, rstd=0, **kw)))


def test_null_descriptors():
    lib = la.load()
    assert lib.la_norm_forward(None, None, None) == INVALID
    assert lib.la_norm_backward(None, None, None, 0, None) == INVALID
    assert lib.la_norm_backward_workspace_bytes(None) == -1
    n = norm()
    assert lib.la_norm_forward(ctypes.byref(n), None, None) == INVALID
    assert lib.la_norm_backward(ctypes.byref(n), None, None, 0, None) == INVALID


def test_nothing_to_do():
    for kw in (dict(outer=0), dict(inner=0), dict(cols=0)):
        la.norm_forward_raw(norm(**kw), forward_io(x=rows(None), y=rows(None), sum=NONE,
                                                   residual=NONE))
        assert la.norm_backward_workspace_bytes_raw(norm(**kw)) == 0
    la.norm_backward_raw(norm(cols=0), backward_io())
    la.norm_backward_raw(norm(outer=0), backward_io(dweight=0, dbias=0))


def test_workspace_by_shapes():
    bf, f32 = torch.bfloat16, torch.float32
    need = la.norm_backward_workspace_bytes
    assert need((4, 8, 100), bf) == need((32, 100), bf)
    assert 2 * 4 * 100 <= need((1, 100), bf) <= need((100000, 100), bf) < 8 * 1025 * 100
    # rows past the registers keep two numbers each
    assert need((7, 16384), bf) < need((7, 16385), bf)
    assert need((7, 8192), f32) < need((7, 8193), f32)
    with pytest.raises(la.LayerAdamError):
        need((3, la.MAX_SIDE + 1), bf)
    with pytest.raises(TypeError):
        need((3, 4), torch.float64)


def test_binding_checks():
    f = torch.zeros
    x = f(4, 6)
    w = f(6)
    stats = f(2, 4)
    cases = [
        (TypeError, lambda: la.layer_norm(f(4, 6, dtype=torch.float64), w)),
        (ValueError, lambda: la.layer_norm(f(()), w)),
        (ValueError, lambda: la.layer_norm(x, f(5))),
        (ValueError, lambda: la.layer_norm(x, f(2, 3))),
        (ValueError, lambda: la.layer_norm(x, f(12)[::2])),
        (TypeError, lambda: la.layer_norm(x, f(6, dtype=torch.int32))),
        (ValueError, lambda: la.layer_norm(x, w, stats=f(1, 4))),
        (ValueError, lambda: la.rms_norm(x, w, stats=f(2, 4))),
        (ValueError, lambda: la.rms_norm(x, w, stats=f(1, 4, dtype=torch.float16))),
        (ValueError, lambda: la.rms_norm(x, w, sum_out=f(4, 6))),
        (ValueError, lambda: la.layer_norm_backward(x, x, w, f(1, 4))),
        (TypeError, lambda: la.layer_norm(x, w)),  # pageable host memory
        (TypeError, lambda: la.layer_norm_backward(x, x, w, stats)),
    ]
    for kind, call in cases:
        with pytest.raises(kind):
            call()
    layout = la._RowLayout(x)
    for bad in (f(4, 7), f(4, 6, dtype=torch.bfloat16), f(6, 4).T):
        with pytest.raises(ValueError):
            layout(bad, "t")
    with pytest.raises(ValueError):  # the axes before the last two are not one stride apart
        la._RowLayout(f(2, 3, 4, 5))(f(3, 2, 4, 5).transpose(0, 1), "t")
    with pytest.raises(TypeError):
        layout.parameter(w.half(), "bias", torch.float32)


@pytest.mark.parametrize("layer", [True, False])
def test_formulas_are_the_derivatives(layer):
    s = inputs(5, 9, torch.float64, 3)
    w, b = params(9, torch.float64, 3)
    dy = inputs(5, 9, torch.float64, 4)
    ds = inputs(5, 9, torch.float64, 5)
    x = s.clone().requires_grad_()
    wg, bg = w.clone().requires_grad_(), b.clone().requires_grad_()
    y, mean, rstd = forward64(x, wg, bg, 1e-5, layer)
    want = torch.autograd.grad((y * dy).sum() + (x * ds).sum(), (x, wg, bg))
    got = backward64(dy, s, w, mean.detach(), rstd.detach(), layer, ds)
    for a, e in zip(got, want):
        assert torch.allclose(a, e, rtol=1e-12, atol=1e-12)
    # against differences: central ones of step 1e-5 are off by about 1e-10
    for i, j in ((0, 0), (2, 5), (4, 8)):
        value = []
        for sign in (1, -1):
            t = s.clone()
            t[i, j] += sign * 1e-5
            value.append((forward64(t, w, b, 1e-5, layer)[0] * dy).sum() + (t * ds).sum())
        assert abs(float(value[0] - value[1]) / 2e-5 - float(got[0][i, j])) < 1e-6
