"""The linear cross entropy in workspaces of other sizes than its own: of a larger
batch, and of every amount between the least that serves and what it asks for;
against the formulas in 64 bits."""
import pytest
import torch

import optimizer_step_layeradam_amd as la
from losshelpers import Truth, problem

pytestmark = pytest.mark.gpu
BF, H = torch.bfloat16, torch.float16


def run(x, w, y, size):
    """All outputs from a workspace of `size` bytes, behind which nothing is written."""
    ws = torch.full((size + 4096,), 165, dtype=torch.uint8, device="cuda")
    losses = torch.empty(y.numel(), device="cuda")
    loss, dx, dw = la.linear_cross_entropy_gradients(x, w, y, reduction="sum", losses=losses,
                                                     workspace=ws[:size])
    assert bool((ws[size:] == 165).all())
    return loss, losses, dx, dw


@pytest.mark.parametrize("dtype", [BF, H])
@pytest.mark.parametrize("tokens,larger,hidden,vocab", [
    (1, 20, 64, 3000), (20, 65, 320, 5000), (64, 100, 200, 5000), (300, 330, 320, 5000),
    (640, 641, 256, 2100), (1300, 1400, 576, 1030), (2050, 2300, 128, 900)])
def test_of_a_larger_batch(tokens, larger, hidden, vocab, dtype):
    x, w, y = (t.cuda() for t in problem(tokens, hidden, vocab, dtype, 41, 0.2))
    truth = Truth(x, w, y, mean=False)
    for columns in (0, 512):
        size = la.linear_cross_entropy_workspace_bytes(larger, hidden, vocab,
                                                       piece_columns=columns)
        truth.check(*run(x, w, y, size))
    size = la.linear_cross_entropy_workspace_bytes(larger, hidden, vocab, input_grad=False,
                                                   weight_grad=False)
    losses = torch.empty(tokens, device="cuda")
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    truth.check(la.linear_cross_entropy(x, w, y, reduction="sum", losses=losses, workspace=ws),
                losses)


@pytest.mark.parametrize("tokens,hidden,vocab", [(24, 512, 9000), (300, 320, 5000),
                                                 (2050, 320, 2100)])
def test_between_least_and_most(tokens, hidden, vocab):
    x, w, y = (t.cuda() for t in problem(tokens, hidden, vocab, BF, 42, 0.1))
    truth = Truth(x, w, y, mean=False)
    least, most = (la.linear_cross_entropy_workspace_bytes(tokens, hidden, vocab, piece_columns=c)
                   for c in (1, 0))
    for k in range(9):
        size = least + (most - least) * k // 8
        truth.check(*run(x, w, y, size))


@pytest.mark.parametrize("dtype", [BF, H])
def test_large_tiles_in_pieces(dtype):
    """Products of 256 x 256 tiles over several pieces, the last one shorter: the
    workspace holds less than the whole matrix."""
    tokens, hidden, vocab = 2310, 4160, 18000
    size = 2 * tokens * vocab
    assert size > la.linear_cross_entropy_workspace_bytes(tokens, hidden, vocab, piece_columns=1)
    x, w, y = (t.cuda() for t in problem(tokens, hidden, vocab, dtype, 43, 0.1))
    Truth(x, w, y, mean=False).check(*run(x, w, y, size))
