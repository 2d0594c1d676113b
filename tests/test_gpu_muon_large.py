"""Stacks of more than 2^32 elements, in each form: the last matrix, whose
offsets pass 32 bits, against the polynomial in 64 bits, and the first."""
import pytest
import torch

import optimizer_step_layeradam_amd as la
from muonhelpers import DIRECTION, HALF_STEP, direction64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(70000, 16, 4000), (511, 16, 550000), (17000, 64, 4000),
                                   (511, 66000, 128), (257, 4096, 4096)], ids=str)
def test_offsets_past_32_bits(shape):
    assert shape[0] * shape[1] * shape[2] > 2 ** 32
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for part in x.split(max(1, shape[0] // 64)):
        part.normal_(generator=gen)
    o = torch.zeros_like(x)
    la.orthogonalize(x, o)
    for z in (0, shape[0] // 2, -1):
        want = direction64(x[z])
        d = float((o[z].double() - want).norm() / want.norm())
        print(f"  {shape} matrix {z}: {d:.2e}", flush=True)
        assert d <= DIRECTION + HALF_STEP[torch.bfloat16]
    del x, o
    torch.cuda.empty_cache()
