"""Kernels that start before the one before them has ended (kivi_launch_after) read
global memory by ordinary loads only."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_kv_quantize_gb300", "csrc")


def test_no_read_only_loads():
    files = [f for f in glob.glob(os.path.join(CSRC, "*.cu")) if "kivi_launch_after(" in open(f).read()]
    assert len(files) >= 4
    for f in files:
        code = re.sub(r"//.*", "", open(f).read())
        assert not re.search(r"__restrict__|__ldg\b|\.nc\b|ld\.global\.nc", code), os.path.basename(f)
