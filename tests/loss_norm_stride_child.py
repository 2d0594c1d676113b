"""Run by test_gpu_loss_large.py with a capped grid: every kernel of the linear
cross entropy and of the norms strides over its work, with the same bits."""
import os
import sys

import torch

sys.path[:0] = [os.path.dirname(os.path.abspath(__file__)),
                os.path.dirname(os.path.dirname(os.path.abspath(__file__)))]
import optimizer_step_layeradam_amd as la  # noqa: E402
from losshelpers import problem  # noqa: E402
from normhelpers import inputs, params  # noqa: E402

out = []
for tokens, hidden, vocab, columns in ((20, 192, 3000, 0), (50, 100, 3000, 512),
                                       (300, 320, 5000, 1024), (2100, 96, 300, 0),
                                       (2049, 640, 8200, 4096)):
    x, w, y = (t.cuda() for t in problem(tokens, hidden, vocab, torch.bfloat16, 1, 0.2))
    need = la.linear_cross_entropy_workspace_bytes(tokens, hidden, vocab, piece_columns=columns)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    losses = torch.empty(tokens, device="cuda")
    out += [losses, *la.linear_cross_entropy_gradients(x, w, y, losses=losses, workspace=ws)]
    print("loss", tokens, hidden, vocab, flush=True)
for rows, cols in ((9, 5), (700, 33), (5000, 128), (300, 3000), (40, 5121), (60, 20000)):
    x, dy = inputs(rows, cols, torch.bfloat16, 1).cuda(), inputs(rows, cols, torch.bfloat16, 2).cuda()
    w, b = (t.cuda() for t in params(cols, torch.float32))
    y, stats, s = la.layer_norm(x, w, b, residual=dy)
    out += [y, stats, s, *la.layer_norm_backward(dy, s, w, stats)]
    print("norm", rows, cols, flush=True)
torch.save([t.cpu() for t in out], sys.argv[1])
