"""Rules that the kernels' sources keep, where no run could show a breach."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_epilogue_tmem_gb300", "csrc")


@pytest.mark.parametrize("name", ["k_moe.cu", "fp8.cuh", "fp8_common.cuh", "k_fp8_narrow.cu", "k_fp8_single.cu", "k_fp8_wide.cu"])
def test_no_read_only_loads(name):
    """These kernels are launched while the one that writes their inputs may still run: loads through the read-only
    path, which need data that nobody writes while the kernel lives, are not for them."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in code, word
