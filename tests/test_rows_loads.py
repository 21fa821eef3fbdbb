"""How the kernels of 8-bit rows read memory (no GPU needed).

They begin while the kernel ahead of them, which writes what they read, may still run.  Waiting for it orders ordinary
loads; loads that promise constant memory (ld.global.nc, __ldg, const __restrict__) may be made before, or answered
from what an earlier kernel left in a cache."""
import glob
import os
import re

import pytest

from speculative_decoding_verification_45_gb300 import _native

SOURCES = sorted(glob.glob(os.path.join(_native.ROWS, "*.cu")) + glob.glob(os.path.join(_native.ROWS, "*.cuh")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_promises_constant_memory(path):
    with open(path) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    found = re.findall(r"__ldg|\bld\.(?:weak\.)?global[\w.:]*\.nc\b|__restrict__|__ldcs|\bldu\b", code)
    assert not found


def test_every_source_is_looked_at():
    assert {os.path.basename(p) for p in SOURCES} >= {"spec_rows.cuh", "spec_rows_code.cu", "spec_rows_product.cu"}
