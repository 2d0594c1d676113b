"""What the compiler made of the narrow forms' kernels: no scratch memory, and
no more scalar registers spilled than they have now (their loops over X keep
strides, ends and places of several matrices)."""
import os
import re
import tempfile

import pytest

from test_isa_cpu import _compile, kernel_descriptors


@pytest.fixture(scope="module")
def listing():
    with tempfile.TemporaryDirectory() as d:
        path = os.path.join(d, "narrow.s")
        p = _compile("la_narrow.hip", path)
        log, _ = p.communicate(timeout=600)
        assert p.returncode == 0, log[-3000:]
        with open(path) as f:
            yield f.read()


def test_no_scratch(listing):
    descs = kernel_descriptors(listing)
    assert any("narrow_kernel" in n for n in descs) and any("tiny_kernel" in n for n in descs)
    for name, d in descs.items():
        assert d["amdhsa_private_segment_fixed_size"] == "0", name


def test_spilled_registers(listing):
    """From the kernels' metadata. A spilled scalar is a lane of a vector register
    (v_writelane, v_readlane), a spilled vector would be scratch memory."""
    kernels = re.findall(r"\.name:\s+(\S+)(.*?)\.vgpr_spill_count:\s+(\d+)", listing, re.S)
    assert kernels
    for name, body, vectors in kernels:
        scalars = int(re.search(r"\.sgpr_spill_count:\s+(\d+)", body).group(1))
        assert int(vectors) == 0, name
        assert scalars <= (0 if "tiny_kernel" in name else 144), (name, scalars)


def test_tiny_products_in_binary64(listing):
    assert "v_mfma_f64_16x16x4_f64" in listing
