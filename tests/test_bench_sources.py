"""A recorded capture lapses with any of the kernel's code: the sources that the
bench hashes for a kernel hold every header that they include."""
import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "mxfp8_block_scaled_quantize_gb300", "csrc")


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_included_headers_are_hashed(kernel):
    listed = bench.KERNEL_SOURCES[kernel]
    for f in listed:
        with open(os.path.join(CSRC, f)) as fh:
            included = re.findall(r'#include "([^"/]+\.cuh)"', fh.read())
        assert set(included) <= set(listed), f
