"""Without FP8W_FLAG_WEIGHTS_READY the scales, blocks and bias of a linear layer may be
written by the kernel ahead of it in the stream, which still runs when skinny.cu and
prefill.cu start (programmatic dependent launch).  Their wait for it orders ordinary
loads; a read-only load, which a const __restrict__ pointer allows too, is for memory
that nobody writes while the kernel runs."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_weight_only_gb300", "csrc")


@pytest.mark.parametrize("name", ["skinny.cu", "prefill.cu"])
def test_no_read_only_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert re.findall(r"__ldg|\bldg_stream_\w+|ld\.global\.nc|const\s+\w+\s*\*\s*__restrict__", text) == []
