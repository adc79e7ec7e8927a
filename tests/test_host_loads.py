"""A rule of the kernel sources, checked in the text: kernels launched programmatically run while the
kernel before them still writes, and read-only loads are not ordered behind the wait for it."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "prefix_shared_kv_token_gb300", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h")))


@pytest.mark.parametrize("name", SOURCES)
def test_no_load_takes_the_read_only_path(name):
    """No __ldg or ld.global.nc, and no const __restrict__ pointer, whose loads the compiler may make one."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    found = re.findall(r"__ldg|ld\.global[.\w]*\.nc|__restrict__", code)
    assert not found, found
