"""The orthogonalised update on the host: argument checks of the C ABI and of
the binding, workspace sizes, and the plain form that the GPU tests compare
with against the polynomial of the singular values. No kernel runs here.

The calls with made-up device addresses are all invalid on purpose and must be
refused on the host; they are skipped where a GPU is visible, so that no such
address can reach a device.
"""
import ctypes
import math

import pytest
import torch

import optimizer_step_layeradam_amd as la
from muonhelpers import QUINTIC, direction64, matrices

host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="uses made-up device addresses; host-only check")

BASE = 0x7F0000000000
WS = BASE + 0x7000000000
BIG = 1 << 40
OK, INVALID, MISALIGNED, ALIASING, UNSUPPORTED = 0, 1, 2, 3, 4


def matrix(k=0, rows=40, cols=60, **kw):
    return dict(dict(in_=BASE + k * 0x10000000, out=BASE + 0x1000000000 + k * 0x10000000,
                     rows=rows, cols=cols), **kw)


def refused(status, matrices=None, in_type=la.TYPE_BF16, out_type=la.TYPE_BF16, polynomial=None,
            ws=WS, ws_bytes=BIG):
    desc, keep = la.make_matrices([matrix()] if matrices is None else matrices, in_type, out_type)
    with pytest.raises(la.LayerAdamError) as e:
        la.orthogonalize_raw(desc, polynomial, ws, ws_bytes)
    assert e.value.status == status, str(e.value)
    assert la.last_error()


def test_structs_have_the_sizes_of_the_header():
    import os
    import subprocess
    import tempfile
    names = {"la_polynomial": la.Polynomial, "la_matrix_desc": la.MatrixDesc,
             "la_matrices_desc": la.MatricesDesc, "la_muon_tensor_desc": la.MuonTensorDesc,
             "la_muon_layer_desc": la.MuonLayerDesc, "la_muon_params": la.MuonParams}
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
    (dict(in_type=3), UNSUPPORTED), (dict(in_type=-1), UNSUPPORTED),
    (dict(out_type=la.TYPE_FP32), UNSUPPORTED), (dict(out_type=7), UNSUPPORTED),
    (dict(matrices=[matrix(in_=0)]), INVALID), (dict(matrices=[matrix(out=0)]), INVALID),
    (dict(matrices=[matrix(in_=BASE + 1)]), MISALIGNED),
    (dict(matrices=[matrix(out=BASE + 0x1000000001)]), MISALIGNED),
    (dict(matrices=[matrix(in_=BASE + 2)], in_type=la.TYPE_FP32), MISALIGNED),
    (dict(matrices=[matrix(rows=-1)]), INVALID),
    (dict(matrices=[matrix(cols=la.MAX_SIDE + 1)]), INVALID),
    (dict(matrices=[matrix(count=-2)]), INVALID),
    (dict(matrices=[matrix(rows=la.MAX_SIDE, cols=la.MAX_SIDE, count=1 << 10)]), INVALID),
    (dict(matrices=[matrix(in_row_stride=59)]), INVALID),
    (dict(matrices=[matrix(in_row_stride=-60)]), INVALID),
    (dict(matrices=[matrix(out_row_stride=0)]), INVALID),
    (dict(matrices=[matrix(count=2, in_matrix_stride=40 * 60 - 1)]), INVALID),
    (dict(matrices=[matrix(count=2, in_matrix_stride=60)]), INVALID),
    (dict(matrices=[matrix(count=2, out_row_stride=119, out_matrix_stride=60)]), INVALID),
    (dict(matrices=[matrix(count=2, in_matrix_stride=1 << 62)]), INVALID),
    (dict(matrices=[matrix(in_row_stride=1 << 62)]), INVALID),
    (dict(ws=0), INVALID), (dict(ws=WS + 128), MISALIGNED), (dict(ws_bytes=100), INVALID),
    (dict(ws_bytes=-1), INVALID),
    (dict(ws=BASE), ALIASING), (dict(ws=BASE + 0x1000000000), ALIASING),
    (dict(matrices=[matrix(0), matrix(1, out=BASE + 0x1000000000 + 4798)]), ALIASING),
    (dict(matrices=[matrix(0, out=BASE + 4798)]), ALIASING),
    (dict(matrices=[matrix(0, out=BASE)], in_type=la.TYPE_FP16), ALIASING),
    (dict(matrices=[matrix(0, out=BASE, out_row_stride=61)]), ALIASING),
    (dict(matrices=[matrix(0, out=BASE, count=2, in_matrix_stride=2400,
                           out_matrix_stride=2402)]), ALIASING),
    (dict(matrices=[matrix(0), matrix(1, in_=BASE + 0x1000000000)]), ALIASING),
])
def test_orthogonalize_refuses(kw, status):
    refused(status, **kw)


@host_only
@pytest.mark.parametrize("coefficients,eps", [
    ((), 1e-7), (((1.0, 0.0, 0.0),) * 17, 1e-7), (QUINTIC, -1.0), (QUINTIC, float("nan")),
    (QUINTIC, float("inf")), (((float("nan"), 0.0, 0.0),), 1e-7),
    (((1.0, float("inf"), 0.0),), 1e-7), (((2.0 ** 21, 0.0, 0.0),), 1e-7),
    (((2.0 ** -21, 0.0, 0.0),), 1e-7), (((0.0, 0.0, 0.0),), 1e-7),
    (((200.0, 0.0, 0.0),) * 3, 1e-7),                 # grows step by step
    (((1.0, 2.0 ** 41, -2.0 ** 41),), 1e-7),          # large inside, 1 at the end
])
def test_orthogonalize_refuses_polynomials(coefficients, eps):
    refused(INVALID, polynomial=la.make_polynomial(coefficients, eps))


def test_null_descriptors():
    lib = la.load()
    assert lib.la_orthogonalize(None, None, None, 0, None) == INVALID
    assert lib.la_orthogonalize_workspace_bytes(None, None) == -1
    assert lib.layer_muon_step(None, None, None, None, None, 0, None) == INVALID
    assert lib.layer_muon_workspace_bytes(None, None) == -1
    p = la.Polynomial(None, 5, 1e-7)
    desc, keep = la.make_matrices([], la.TYPE_BF16, la.TYPE_BF16)
    assert lib.la_orthogonalize(ctypes.byref(desc), ctypes.byref(p), None, 0, None) == INVALID


def test_nothing_to_do_needs_no_workspace():
    for xs in ([], [matrix(rows=0)], [matrix(cols=0, in_=0, out=0)], [matrix(count=0)]):
        desc, keep = la.make_matrices(xs, la.TYPE_BF16, la.TYPE_BF16)
        assert la.orthogonalize_workspace_bytes_raw(desc) == 0
        la.orthogonalize_raw(desc)


def muon_tensor(k=0, rows=40, cols=60, R=2, **kw):
    b = BASE + k * 0x100000000
    return dict(dict(master=b, momentum=b + 0x10000000, weight_out=b + 0x20000000,
                     grads=[b + 0x30000000 + r * 0x1000000 for r in range(R)], rows=rows,
                     cols=cols), **kw)


def muon_refused(status, tensors=None, R=2, grad_dtype=la.GRAD_BF16, out_dtype=la.OUT_BF16,
                 flag=0, skip=0, ws=WS, ws_bytes=BIG, raw=None, **hp):
    desc, keep = la.make_muon_layer([muon_tensor()] if tensors is None else tensors, R,
                                    grad_dtype, out_dtype)
    params = la.make_muon_params(**dict(dict(lr=1e-3), **hp))
    for k, v in (raw or {}).items():
        setattr(params, k, v)
    with pytest.raises(la.LayerAdamError) as e:
        la.muon_step_raw(desc, params, flag, skip, ws, ws_bytes)
    assert e.value.status == status, str(e.value)


@host_only
@pytest.mark.parametrize("kw,status", [
    (dict(R=0), INVALID), (dict(R=9), INVALID), (dict(grad_dtype=2), UNSUPPORTED),
    (dict(out_dtype=3), UNSUPPORTED), (dict(lr=-1.0), INVALID), (dict(lr=math.inf), INVALID),
    (dict(momentum=1.0), INVALID), (dict(momentum=-0.1), INVALID),
    (dict(momentum=math.nan), INVALID), (dict(weight_decay=-1e-3), INVALID),
    (dict(grad_unscale=0.0), INVALID), (dict(grad_unscale=math.nan), INVALID),
    (dict(raw=dict(nesterov=2)), INVALID), (dict(raw=dict(lr_scale=3)), UNSUPPORTED),
    (dict(tensors=[muon_tensor(rows=-1)]), INVALID),
    (dict(tensors=[muon_tensor(master=0)]), INVALID),
    (dict(tensors=[muon_tensor(momentum=0)]), INVALID),
    (dict(tensors=[muon_tensor(weight_out=0)]), INVALID),
    (dict(tensors=[muon_tensor(grads=[BASE + 0x30000000, 0])]), INVALID),
    (dict(tensors=[muon_tensor(master=BASE + 4)]), MISALIGNED),
    (dict(tensors=[muon_tensor(grads=[BASE + 0x30000000, BASE + 0x31000008])]), MISALIGNED),
    (dict(tensors=[muon_tensor(momentum=BASE + 9584)]), ALIASING),
    (dict(tensors=[muon_tensor(count=3, momentum=BASE + 3 * 9600 - 16)]), ALIASING),
    (dict(tensors=[muon_tensor(weight_out=BASE + 0x30000000)]), ALIASING),
    (dict(tensors=[muon_tensor(0), muon_tensor(1, master=BASE + 16)]), ALIASING),
    (dict(flag=BASE + 0x40000001), MISALIGNED), (dict(skip=BASE + 0x40000002), MISALIGNED),
    (dict(flag=BASE + 4), ALIASING), (dict(skip=BASE + 4), ALIASING),
    (dict(flag=BASE + 0x40000000, skip=BASE + 0x40000000), ALIASING),
    (dict(flag=WS + 64), ALIASING), (dict(skip=WS + 64), ALIASING),
    (dict(ws=BASE), ALIASING), (dict(ws=0), INVALID), (dict(ws=WS + 16), MISALIGNED),
    (dict(ws_bytes=1000), INVALID),
    (dict(polynomial=la.make_polynomial(((0.0, 0.0, 0.0),))), INVALID),
])
def test_muon_refuses(kw, status):
    muon_refused(status, **kw)


@host_only
def test_muon_many_tensors():
    muon_refused(INVALID, tensors=[muon_tensor(k, 2, 2) for k in range(257)])


def test_workspace_of_a_step():
    def need(nesterov, steps, shape=(400, 600)):
        desc, keep = la.make_muon_layer([dict(rows=shape[0], cols=shape[1])], 1, 0)
        hp = la.make_muon_params(0.0, nesterov=nesterov,
                                 polynomial=la.make_polynomial(((1.5, -0.5, 0.0),) * steps))
        return la.muon_workspace_bytes_raw(desc, hp)

    assert 0 < need(False, 1) < need(False, 2) < need(False, 3) == need(False, 16)
    assert need(True, 1) > need(False, 1)
    # a narrow matrix keeps its FP32 direction at most; a long one also sums of its S
    assert 4 * 40 * 60 <= need(True, 5, (40, 60)) < 4 * 40 * 60 + 1024 > need(False, 5, (40, 60))
    assert need(False, 5, (9000, 40)) > need(False, 5, (500, 40))
    # large matrices: no more than six padded 16-bit copies and two Gram matrices
    assert need(True, 5, (4096, 4096)) < 8.01 * 2 * 4096 ** 2


def test_workspace_by_shapes():
    assert la.orthogonalize_workspace_bytes([(3, 400, 600)]) > \
        la.orthogonalize_workspace_bytes([(400, 600)])
    with pytest.raises(la.LayerAdamError):
        la.orthogonalize_workspace_bytes([(-1, 4)])


def test_binding_checks():
    f = torch.zeros
    with pytest.raises(TypeError):
        la.orthogonalize(f(4, 4, dtype=torch.float64))
    with pytest.raises(TypeError):
        la.orthogonalize([f(4, 4), f(4, 4, dtype=torch.bfloat16)])
    with pytest.raises(TypeError):
        la.orthogonalize(f(4, 4), f(4, 4))
    with pytest.raises(ValueError):
        la.orthogonalize(f(4))
    with pytest.raises(ValueError):
        la.orthogonalize(f(4, 4), f(4, 5, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        la.orthogonalize(f(4, 4, 2)[..., 0])
    with pytest.raises(ValueError):
        la.orthogonalize(f(4, 6), f(6, 4, dtype=torch.bfloat16).mT)
    with pytest.raises(ValueError):
        la.orthogonalize([f(4, 4)], [])
    with pytest.raises(TypeError):
        la.orthogonalize(f(4, 4))  # pageable host memory
    with pytest.raises(ValueError):
        la.make_polynomial(((1.0, 2.0),))
    with pytest.raises(ValueError):
        la.make_muon_params(1.0, lr_scale="rms")
    g = [f(4, 4, dtype=torch.bfloat16)]
    with pytest.raises(ValueError):
        la.MuonLayer([(f(16), f(16), None)], [g])
    with pytest.raises(TypeError):
        la.MuonLayer([(f(4, 4, dtype=torch.float64), f(4, 4), None)], [g])
    with pytest.raises(ValueError):
        la.MuonLayer([(f(4, 4), f(4, 5), None)], [g])
    with pytest.raises(ValueError):
        la.MuonLayer([(f(4, 4), f(4, 4), None)], [])
    with pytest.raises(ValueError):
        la.MuonLayer([(f(4, 4), f(4, 4), None)], [g * 9])


@pytest.mark.parametrize("shape", [(7, 12), (12, 7), (2, 9, 9)])
def test_plain_form_is_the_polynomial_of_the_singular_values(shape):
    u = matrices(shape, seed=1).double()
    a, s, b = torch.linalg.svd(u, full_matrices=False)
    s = s / s.norm(dim=-1, keepdim=True)
    for k1, k3, k5 in QUINTIC:
        s = k1 * s + k3 * s ** 3 + k5 * s ** 5
    want = a @ torch.diag_embed(s) @ b
    assert torch.allclose(direction64(u), want, rtol=0, atol=1e-11)
