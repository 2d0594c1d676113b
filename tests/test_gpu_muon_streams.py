"""The memory that orthogonalize() hands out belongs to the stream that writes
it: a block that work on another stream may still use is not taken, nor given
back to that stream while the writing stream may still be at it."""
import pytest
import torch

import optimizer_step_layeradam_amd as la
from muonhelpers import matrices

pytestmark = pytest.mark.gpu


def test_default_output_on_another_stream():
    x = matrices((300, 500), seed=1).cuda()
    want = la.orthogonalize(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    before = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
    freed = before.data_ptr()  # on the current stream, as after work that is still pending there
    del before
    o = la.orthogonalize(x, stream=s)
    assert o.data_ptr() != freed
    s.synchronize()
    assert torch.equal(o.view(torch.int16), want.view(torch.int16))
    written = o.data_ptr()
    del o
    after = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
    assert after.data_ptr() != written
