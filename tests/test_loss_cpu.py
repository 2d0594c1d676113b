"""The linear cross entropy on the host: argument checks of the C ABI and of
the binding, workspace sizes, and the formulas that the GPU tests compare with
against differentiation and against differences. No kernel runs here.

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
from losshelpers import Truth, problem

host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="uses made-up device addresses; host-only check")

BASE = 0x7F0000000000
STEP = 0x1000000000
WS = BASE + 0x100 * STEP
BIG = 1 << 40
INVALID, MISALIGNED, ALIASING, UNSUPPORTED = 1, 2, 3, 4
T, H, V = 50, 128, 1000


def at(k, offset=0):
    return BASE + k * STEP + offset


def desc(**kw):
    d = dict(x=at(0), weight=at(1), targets=at(2), tokens=T, hidden=H, vocab=V,
             type=la.TYPE_BF16, target_type=la.INDEX_INT64, reduction=0, loss=at(3),
             losses=at(4), dx=at(5), dweight=at(6))
    d.update(kw)
    return la.make_cross_entropy(**d)


def refuses(status, d, ws=WS, size=BIG):
    with pytest.raises(la.LayerAdamError) as e:
        la.linear_cross_entropy_raw(d, ws, size)
    assert e.value.status == status, str(e.value)
    assert la.last_error()


def test_struct_has_the_size_of_the_header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with tempfile.TemporaryDirectory() as d:
        src = os.path.join(d, "t.c")
        with open(src, "w") as f:
            f.write('#include "layeradam.h"\n#include <stdio.h>\nint main(void){'
                    'printf("%zu\\n", sizeof(la_cross_entropy_desc));return 0;}\n')
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), src, "-o",
                        os.path.join(d, "t")], check=True)
        size = subprocess.run([os.path.join(d, "t")], capture_output=True, text=True,
                              check=True).stdout
    assert int(size) == ctypes.sizeof(la.CrossEntropyDesc)


@host_only
@pytest.mark.parametrize("kw,status", [
    (dict(type=la.TYPE_FP32), UNSUPPORTED), (dict(type=-1), UNSUPPORTED),
    (dict(target_type=2), UNSUPPORTED), (dict(reduction=2), UNSUPPORTED),
    (dict(tokens=-1), INVALID), (dict(hidden=0), INVALID), (dict(vocab=0), INVALID),
    (dict(tokens=la.MAX_SIDE + 1), INVALID), (dict(vocab=la.MAX_SIDE + 1), INVALID),
    (dict(hidden=la.MAX_SIDE + 1), INVALID),
    (dict(grad_scale=float("nan")), INVALID), (dict(grad_scale=float("inf")), INVALID),
    (dict(grad_scale=1e39), INVALID), (dict(grad_scale=-1e300), INVALID),
    (dict(x_row_stride=-1), INVALID), (dict(x_row_stride=1 << 41), INVALID),
    (dict(weight_row_stride=H - 1), INVALID), (dict(dx_row_stride=0), INVALID),
    (dict(dweight_row_stride=H - 1), INVALID), (dict(dweight_row_stride=1 << 41), INVALID),
    (dict(x=0), INVALID), (dict(weight=0), INVALID), (dict(targets=0), INVALID),
    (dict(loss=0), INVALID),
    (dict(x=at(0, 1)), MISALIGNED), (dict(weight=at(1, 1)), MISALIGNED),
    (dict(targets=at(2, 4)), MISALIGNED),
    (dict(targets=at(2, 2), target_type=la.INDEX_INT32), MISALIGNED),
    (dict(loss=at(3, 2)), MISALIGNED), (dict(losses=at(4, 1)), MISALIGNED),
    (dict(dx=at(5, 1)), MISALIGNED), (dict(dweight=at(6, 1)), MISALIGNED),
    (dict(dx=at(0)), ALIASING), (dict(dx=at(0, 2 * (T * H - 1))), ALIASING),
    (dict(dweight=at(1)), ALIASING), (dict(dweight=at(5, 2 * (T * H - 1))), ALIASING),
    (dict(losses=at(3, 0)), ALIASING), (dict(loss=at(2, 8)), ALIASING),
    (dict(loss=at(4, 4 * (T - 1))), ALIASING), (dict(dx=WS + 1024), ALIASING),
    (dict(x=WS), ALIASING),
])
def test_refuses(kw, status):
    refuses(status, desc(**kw))


@host_only
def test_refuses_workspaces():
    least = la.linear_cross_entropy_workspace_bytes_raw(desc(), 1)
    assert least > 0
    refuses(INVALID, desc(), 0)
    refuses(MISALIGNED, desc(), WS + 128)
    refuses(INVALID, desc(), WS, least - 1)
    refuses(INVALID, desc(), WS, -1)
    refuses(ALIASING, desc(), at(6))
    # without gradients less is enough, and that less is checked too
    none = desc(dx=0, dweight=0)
    need = la.linear_cross_entropy_workspace_bytes_raw(none)
    assert 0 < need < least
    refuses(INVALID, none, WS, need - 1)


def test_null_descriptors():
    lib = la.load()
    assert lib.la_linear_cross_entropy(None, None, 0, None) == INVALID
    assert lib.la_linear_cross_entropy_workspace_bytes(None, 0) == -1


def test_workspace_by_shapes():
    need = la.linear_cross_entropy_workspace_bytes
    whole = need(8192, 5120, 150000)
    # one piece of the whole vocabulary, and little beside it
    assert 2 * 8192 * 150000 < whole < 2 * 8192 * 150000 + (1 << 30)
    # not more than 4 GiB of pieces however many tokens there are
    assert need(1 << 20, 64, 150000) < (4 << 30) + 9 * (1 << 20) * 150000 // 64 + (1 << 30)
    sizes = [need(1000, 512, 50000, piece_columns=c) for c in (1, 256, 1000, 25000, 50000, 10 ** 9)]
    assert sizes[0] == sizes[1] < sizes[2] < sizes[3] < sizes[4] == sizes[5]
    assert need(1000, 512, 50000, weight_grad=False, input_grad=False) < sizes[0]
    # rows that are no whole depth, or not aligned, are copied
    assert need(10, 513, 50000) > need(10, 512, 50000) + 2 * 50000 * 513
    assert need(10, 512, 50000, packed=True) >= need(10, 512, 50000) + 2 * 50000 * 512
    assert 0 < need(0, 512, 50000) < need(1, 512, 50000)
    for bad in ((-1, 4, 4), (4, 0, 4), (4, 4, la.MAX_SIDE + 1)):
        with pytest.raises(la.LayerAdamError):
            need(*bad)
    with pytest.raises(la.LayerAdamError):
        need(4, 4, 4, piece_columns=-1)


def test_binding_checks():
    bf = torch.bfloat16
    x, w, y = torch.zeros(4, 6, dtype=bf), torch.zeros(9, 6, dtype=bf), torch.zeros(4).long()
    f = la.linear_cross_entropy_gradients
    cases = [
        (ValueError, lambda: f(x, w, y, reduction="none")),
        (ValueError, lambda: f(x, w[0], y)),
        (TypeError, lambda: f(x.float(), w.float(), y)),
        (TypeError, lambda: f(x, w.half(), y)),
        (TypeError, lambda: f(x, w, y.float())),
        (ValueError, lambda: f(x, w, y[:3])),
        (ValueError, lambda: f(x, w, torch.zeros(8).long()[::2])),
        (ValueError, lambda: f(x, torch.zeros(9, 7, dtype=bf), y)),
        (ValueError, lambda: f(x, w, y, loss=torch.zeros(2))),
        (ValueError, lambda: f(x, w, y, loss=torch.zeros((), dtype=torch.float64))),
        (ValueError, lambda: f(x, w, y, losses=torch.zeros(5))),
        (ValueError, lambda: f(torch.zeros(6, 4, dtype=bf).T, w, y)),
        (ValueError, lambda: f(torch.zeros(3, 2, 6, dtype=bf).transpose(0, 1), w,
                               torch.zeros(2, 3).long())),
        (TypeError, lambda: f(x, w, y)),  # pageable host memory
    ]
    for kind, call in cases:
        with pytest.raises(kind):
            call()
    with pytest.raises(ValueError):
        la._check_matrix(torch.zeros(4, 5, dtype=bf), (4, 6), bf, "dx")


def test_formulas_are_the_derivatives():
    x, w, y = problem(9, 12, 30, torch.bfloat16, 3, 0.3)
    t = Truth(x, w, y, mean=True, scale=2.0)
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    loss = torch.nn.functional.cross_entropy(xd @ wd.T, y, ignore_index=-100)
    dx, dw = torch.autograd.grad(2.0 * loss, (xd, wd))
    assert abs(float(loss.detach() - t.loss)) < 1e-12
    assert torch.allclose(t.dx, dx, atol=1e-13) and torch.allclose(t.dw, dw, atol=1e-13)
    # against differences: central ones of step 1e-5 are off by about 1e-10
    for a, i, j, g in ((xd, 1, 5, t.dx), (wd, 7, 3, t.dw), (wd, int(y[y >= 0][0]), 0, t.dw)):
        value = []
        for sign in (1, -1):
            with torch.no_grad():
                a[i, j] += sign * 1e-5
                value.append(torch.nn.functional.cross_entropy(xd @ wd.T, y, ignore_index=-100))
                a[i, j] -= sign * 1e-5
        assert abs(2 * float(value[0] - value[1]) / 2e-5 - float(g[i, j])) < 1e-7


def test_truth_without_tokens():
    x, w, y = problem(5, 12, 30, torch.float16, 3, 1.1)
    t = Truth(x, w, y)
    t.check(torch.zeros(()), torch.zeros(5), torch.zeros(5, 12), torch.zeros(30, 12))
