"""Workspaces of the norms' backward pass on the host: which sizes a call takes,
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
STEP = 0x10000000000
INVALID, ALIASING = 1, 3


def at(k):
    return BASE + k * STEP


def takes(rows, cols, dtype, size):
    """Whether a call over these rows takes a workspace of `size` bytes: it is
    checked before the buffers against each other, and dweight is dbias here."""
    def of(k):
        return la.Rows(at(k), cols, 0)

    desc = la.make_norm(la.NORM_LAYER, rows, 1, cols, la._element_types()[dtype], la.TYPE_FP32)
    io = la.NormBackwardIO(of(0), of(1), la.Rows(), of(2), at(3), at(4), at(5), at(5),
                           la.TYPE_FP32)
    with pytest.raises(la.LayerAdamError) as e:
        la.norm_backward_raw(desc, io, at(6), size)
    assert e.value.status in (INVALID, ALIASING), str(e.value)
    return e.value.status == ALIASING


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("cols", [1, 33, 128, 1024, 2560, 4096, 5120, 8192, 12288, 20000, 32768,
                                  32769, 70001])
def test_a_size_serves_fewer_rows(cols, dtype):
    """A workspace that is kept for a batch serves every smaller one."""
    counts = sorted({1, 2, 3, *(n + d for n in (4, 256, 512, 1024, 2048, 4096, 16384, 65536,
                                                1 << 20) for d in (-1, 0, 1)),
                     *range(40, 9000, 347), 2049, 2560, 5000, 32768})
    least = float("inf")
    for rows in reversed(counts):
        size = la.norm_backward_workspace_bytes((rows, cols), dtype)
        least = min(least, size)
        assert takes(rows, cols, dtype, least), (rows, least, size)
        assert not takes(rows, cols, dtype, min(least, size) // 1024)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_rows_past_the_registers_keep_two_numbers_each(dtype):
    """From 32769 elements on; as many parts as there can be at both row counts."""
    need = la.norm_backward_workspace_bytes
    for cols, each in ((8192, 0), (16385, 0), (32768, 0), (32769, 8), (70001, 8)):
        more = need((204800, cols), dtype) - need((102400, cols), dtype)
        assert more == each * 102400, (cols, more)
