"""What the compiler made of the norms' backward kernels, one source an element
type, from their assembly for gfx950: no packed FP32 arithmetic, denormals kept
and rounding to nearest even; and how much of their rows lies in scratch memory,
which is nothing up to 256 lanes a row. Rows of 16 to 32 KB share the 128
registers a lane of a workgroup of 1024 with their parameter and their columns'
sums: 16-bit rows that end inside a vector, with a bias and a residual's gradient,
leave 57 of these in scratch, whole vectors without either 5."""
import os
import re
import tempfile

import pytest

from test_isa_cpu import _compile, kernel_descriptors

TYPES = ("bf16", "fp16", "fp32")


@pytest.fixture(scope="module")
def listings():
    with tempfile.TemporaryDirectory() as d:
        procs = {t: _compile(f"la_norm_backward_{t}.hip", os.path.join(d, t + ".s"))
                 for t in TYPES}
        out = {}
        for t, p in procs.items():
            log, _ = p.communicate(timeout=600)
            assert p.returncode == 0, log[-3000:]
            with open(os.path.join(d, t + ".s")) as f:
                out[t] = f.read()
        yield out


@pytest.mark.parametrize("of", TYPES)
def test_instructions_and_number_modes(listings, of):
    assert not re.findall(r"\bv_pk_(?:add|mul|fma)_f32\b", listings[of])
    for name, d in kernel_descriptors(listings[of]).items():
        assert d["amdhsa_float_denorm_mode_32"] == "3", name
        assert d["amdhsa_float_denorm_mode_16_64"] == "3", name
        assert d["amdhsa_float_round_mode_32"] == "0", name


@pytest.mark.parametrize("of", TYPES)
def test_scratch(listings, of):
    seen = 0
    for name, d in kernel_descriptors(listings[of]).items():
        scratch = int(d["amdhsa_private_segment_fixed_size"])
        if "wide_kernel" in name:
            assert scratch <= 192, (name, scratch)
        elif "ELi1024E" in name:
            whole, fp32 = "EndsE0E" in name, of == "fp32"
            assert scratch <= (0 if whole else 48) if fp32 else (96 if whole else 232), \
                (name, scratch)
            seen += 1
        else:
            assert scratch == 0, (name, scratch)
    assert seen == 8
