"""Run by test_gpu_muon_tiny.py with a capped grid: the kernels of short sides
up to 16 stride over their work."""
import os
import sys

import torch

sys.path[:0] = [os.path.dirname(os.path.abspath(__file__)),
                os.path.dirname(os.path.dirname(os.path.abspath(__file__)))]
import optimizer_step_layeradam_amd as la  # noqa: E402
from muonhelpers import HALF_STEP, direction64, matrices, off  # noqa: E402

for shape in ((40, 5, 9), (9, 16, 16), (3, 7, 1500), (2, 2000, 12)):
    x = matrices(shape, seed=1).cuda()
    o = la.orthogonalize(x, torch.empty(shape, dtype=torch.float16, device="cuda"))
    got = off(o, direction64(x.cpu()))
    print("orthogonalize", shape, f"{got:.2e}", flush=True)
    assert got <= HALF_STEP[torch.float16] + 1.1e-5
    p, m = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
    g = x.to(torch.bfloat16)
    la.muon_step([(p, m, None)], [[g]], lr=1.0, lr_scale="none")
    got = off(-p, direction64(g.cpu()))
    print("muon_step", shape, f"{got:.2e}", flush=True)
    assert got <= 1.1e-5 and torch.equal(m, g.float())
