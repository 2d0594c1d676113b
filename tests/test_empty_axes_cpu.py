"""Tensors without rows as the norms and the linear cross entropy divide them
into rows: torch gives an axis of length 0 the strides of one of length 1, which
are one stride apart all the same, there being no rows. No kernel runs here."""
import pytest
import torch

import optimizer_step_layeradam_amd as la

SHAPES = [(0, 8), (2, 0, 8), (0, 2, 8), (2, 0, 3, 8), (0, 2, 3, 8), (2, 3, 0, 8), (2, 0, 0, 8),
          (5, 2, 0, 3, 8)]


@pytest.mark.parametrize("shape", SHAPES)
def test_rows_of_a_tensor_without_rows(shape):
    t = torch.empty(shape)
    layout = la._RowLayout(t)
    assert layout.rows == 0 and layout(t, "t").data is None
    matrix = la._token_rows(t, "t")
    assert tuple(matrix.shape) == (0, 8)


def test_axes_with_rows_are_still_looked_at():
    for shape in ((2, 3, 4, 8), (1, 2, 3, 4, 8)):
        t = torch.empty(shape)
        la._token_rows(t, "t")
        turned = t.transpose(-4, -3)
        with pytest.raises(ValueError):
            la._token_rows(turned, "t")
        with pytest.raises(ValueError):
            la._RowLayout(turned)(turned, "t")
