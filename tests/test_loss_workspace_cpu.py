"""Workspaces of the linear cross entropy on the host: which sizes a call takes,
asked by calls that are refused for another reason once the size will do. No
kernel runs here.

The calls have made-up device addresses and must be refused on the host; they
are skipped where a GPU is visible, so that no such address can reach a device.
"""
import pytest
import torch

import optimizer_step_layeradam_amd as la

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="uses made-up device addresses; host-only check")

BASE = 0x7F0000000000
STEP = 0x1000000000
INVALID, ALIASING = 1, 3


def takes(tokens, hidden, vocab, size, grads=True):
    """Whether a call of these sizes takes a workspace of `size` bytes: it is
    checked before the buffers against each other, and `loss` lies in the weight."""
    d = la.make_cross_entropy(
        x=BASE, weight=BASE + STEP, targets=BASE + 2 * STEP, tokens=tokens, hidden=hidden,
        vocab=vocab, type=la.TYPE_BF16, target_type=la.INDEX_INT64, reduction=0,
        loss=BASE + STEP, dx=grads and BASE + 4 * STEP, dweight=grads and BASE + 5 * STEP)
    with pytest.raises(la.LayerAdamError) as e:
        la.linear_cross_entropy_raw(d, BASE + 0x100 * STEP, size)
    assert e.value.status in (INVALID, ALIASING), str(e.value)
    return e.value.status == ALIASING


def need(tokens, hidden, vocab, grads=True, columns=0):
    return la.linear_cross_entropy_workspace_bytes(tokens, hidden, vocab, piece_columns=columns,
                                                   input_grad=grads, weight_grad=grads)


def told(tokens, hidden, vocab, size):
    """The least size that a refusal names."""
    with pytest.raises(la.LayerAdamError) as e:
        la.linear_cross_entropy_raw(la.make_cross_entropy(
            x=BASE, weight=BASE + STEP, targets=BASE + 2 * STEP, tokens=tokens, hidden=hidden,
            vocab=vocab, type=la.TYPE_BF16, target_type=la.INDEX_INT64, reduction=0,
            loss=BASE + 3 * STEP, dx=BASE + 4 * STEP, dweight=BASE + 5 * STEP),
            BASE + 0x100 * STEP, size)
    assert e.value.status == INVALID
    return int(str(e.value).rsplit(" ", 1)[1])


SHAPES = [(4096, 128000), (2560, 150000), (8192, 32000), (512, 700), (64, 5000), (2049, 50021)]


@pytest.mark.parametrize("grads", [False, True])
@pytest.mark.parametrize("hidden,vocab", SHAPES)
def test_a_size_serves_fewer_tokens(hidden, vocab, grads):
    """A workspace that is kept for a batch serves every smaller one."""
    counts = sorted({0, 1, 2, *(n + d for n in range(32, 2400, 32) for d in (0, 1)), 641, 1535,
                     1548, 1664, 1665, 4096, 4097, 8191, 8192})
    for columns in (0, 1024) if grads else (0,):
        sizes = [need(t, hidden, vocab, grads, columns) for t in counts]
        # the size of each number of tokens against that of every larger one: the
        # smallest of these is enough to look at
        least = float("inf")
        for t, size in zip(reversed(counts), reversed(sizes)):
            least = min(least, size)
            assert takes(t, hidden, vocab, least, grads), (t, least, size)


@pytest.mark.parametrize("hidden,vocab", SHAPES)
@pytest.mark.parametrize("tokens", [1, 50, 640, 1535, 8192])
def test_a_refusal_names_the_least_that_serves(tokens, hidden, vocab):
    least = told(tokens, hidden, vocab, 0)
    assert takes(tokens, hidden, vocab, least)
    for less in (least - 1, least - 256, least // 2, 1):
        assert not takes(tokens, hidden, vocab, less)
    for more in (least + 1, 2 * least, need(tokens, hidden, vocab), 1 << 44):
        assert takes(tokens, hidden, vocab, max(more, least))


@pytest.mark.parametrize("tokens,hidden,vocab", [
    (8192, 8192, 4000), (8192, 5120, 150000), (2310, 4160, 8200), (24, 4096, 128000),
    (1000, 2048, 30000), (3, 64, 900)])
def test_smaller_pieces_never_need_more(tokens, hidden, vocab):
    """And what they need is taken."""
    columns = sorted({1, 256, 257, 512, 1024, 1280, 2048, 2304, 4000, 4096, 8192, 30000, 50000,
                      75000, 75008, vocab, 1 << 20})
    sizes = [need(tokens, hidden, vocab, columns=c) for c in columns]
    assert sizes == sorted(sizes), list(zip(columns, sizes))
    least = told(tokens, hidden, vocab, 0)
    for size in sizes:
        assert size >= least and takes(tokens, hidden, vocab, size)
