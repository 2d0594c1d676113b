"""The linear cross entropy in its large tiles and in those that short sums and
few words take, and all of its kernels and the norms' under a capped grid."""
import os
import subprocess
import sys

import pytest
import torch

import optimizer_step_layeradam_amd as la
from losshelpers import Truth, problem

pytestmark = pytest.mark.gpu
BF, H = torch.bfloat16, torch.float16


def run(x, w, y, mean, scale, columns=0):
    need = la.linear_cross_entropy_workspace_bytes(*x.shape, w.shape[0], piece_columns=columns)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    losses = torch.empty(y.numel(), device="cuda")
    loss, dx, dw = la.linear_cross_entropy_gradients(
        x, w, y, reduction="mean" if mean else "sum", grad_scale=scale, losses=losses, workspace=ws)
    return loss, losses, dx, dw


@pytest.mark.parametrize("dtype,columns", [(BF, 0), (H, 0), (BF, 4096)])
def test_large_tiles(dtype, columns):
    """All three products in 256 x 256 tiles, none of their sides a multiple."""
    x, w, y = (t.cuda() for t in problem(2310, 4160, 8200, dtype, 1, 0.1))
    Truth(x, w, y, mean=False, scale=0.5).check(*run(x, w, y, False, 0.5, columns))


@pytest.mark.parametrize("dtype", [BF, H])
@pytest.mark.parametrize("tokens,hidden,vocab", [(5000, 64, 70), (3001, 130, 310), (700, 1000, 260),
                                                 (900, 2000, 1000), (66, 4096, 700)])
def test_few_tiles(tokens, hidden, vocab, dtype):
    x, w, y = (t.cuda() for t in problem(tokens, hidden, vocab, dtype, 2, 0.2))
    scale = 64.0 if dtype == H else 1.0
    Truth(x, w, y, mean=True, scale=scale).check(*run(x, w, y, True, scale))


def test_capped_grids(tmp_path):
    here = os.path.dirname(os.path.abspath(__file__))
    got = []
    for cap in ("", "1", "7"):
        env = dict(os.environ)
        if cap:
            env["LAYERADAM_MAX_GRID"] = cap
        path = str(tmp_path / f"out{cap}")
        r = subprocess.run([sys.executable, "-u", os.path.join(here, "loss_norm_stride_child.py"),
                            path], env=env, capture_output=True, text=True, timeout=110)
        assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
        got.append(torch.load(path, weights_only=True))
    for other in got[1:]:
        for p, q in zip(got[0], other):
            assert torch.equal(p, q)
