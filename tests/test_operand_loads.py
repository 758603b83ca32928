"""The kernels of rope.cu and attention*.cu start while those ahead of them in
the stream still write pages, scales, rows and indices (programmatic dependent
launch).  The wait for them orders ordinary loads, and a read-only load is for
memory that nobody writes while the kernel runs: the sources have none.  Of the
linear kernels gemv.cu reads its activations by plain loads; they come from such
a kernel (attention's output, say)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_weight_only_gb300", "csrc")


@pytest.mark.parametrize("name", ["rope.cu", "attention.cuh", "attention.cu", "attention_few.cu"])
def test_no_read_only_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    # ldg_stream_*: the shared header's read-only loads
    assert re.findall(r"__ldg|\bldg_stream_\w+|ld\.global\.nc|__restrict__", text) == []


def test_the_gemv_has_no_read_only_load_of_its_activations():
    with open(os.path.join(CSRC, "gemv.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert re.findall(r"__ldg\s*\(\s*xg|\bldg_stream_\w+\s*\(\s*xg|uint16_t\s*\*\s*__restrict__\s*x\b", text) == []
