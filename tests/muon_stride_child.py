"""Run by test_gpu_orthogonalize.py with a capped grid: every kernel of the
orthogonalised update and the Muon step strides over its work."""
import os
import sys

import torch

sys.path[:0] = [os.path.dirname(os.path.abspath(__file__)),
                os.path.dirname(os.path.dirname(os.path.abspath(__file__)))]
import optimizer_step_layeradam_amd as la  # noqa: E402
from muonhelpers import DIRECTION, HALF_STEP, direction64, matrices, off  # noqa: E402

for shape in ((3, 65, 130), (300, 140), (40, 5, 9), (2, 513, 300)):
    x = matrices(shape, seed=1).cuda()
    got = off(la.orthogonalize(x), direction64(x.cpu()))
    print("orthogonalize", shape, f"{got:.2e}", flush=True)
    assert got <= DIRECTION + HALF_STEP[torch.bfloat16]
    p, m = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
    g = x.to(torch.bfloat16)
    la.muon_step([(p, m, None)], [[g]], lr=1.0, lr_scale="none")
    got = off(-p, direction64(g.cpu()))
    print("muon_step", shape, f"{got:.2e}", flush=True)
    assert got <= DIRECTION and torch.equal(m, g.float())
