"""The dequantising warps of prefill.cu, skinny.cu and attention.cu read codes from a
ring slot that a copy fills again once they have arrived.  An arrival right behind the
loads can overtake them where shared memory is busy (rows of a warp were wrong then), so
it stands behind the stores of what was read: the sources say so.  (A race is no test.)
fp4_linear.cu reads activations that the kernel before it in the stream may still be
writing: by ordinary loads."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_weight_only_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def faults(text):
    """Arrivals on a slot's barrier with loads and no store between them and what was before."""
    marks = re.compile(r"= (?:mine \? )?lds128\(|sts128\(|tmem_st_x8\(|if \(!mine\) \{|if \(j >= nkb\) \{|"
                       r"mbar_arrive\((?:cempty\([^()]*\)|rawempty\([^()]*\)|taken)\)")
    found, last = [], ""
    for m in marks.finditer(text):
        what = m[0]
        if what.startswith("mbar_arrive") and "lds128" in last:
            found.append(what)
        last = what
    return found


def test_the_reader_sees_an_arrival_behind_loads():
    assert faults("c = lds128(x); if (lane == 0) mbar_arrive(cempty(s));")
    assert not faults("c = lds128(x); sts128(y, c); if (lane == 0) mbar_arrive(cempty(s));")
    assert not faults("c = mine ? lds128(x) : z; if (!mine) { mbar_arrive(cempty(s)); continue; } sts128(y); mbar_arrive(cempty(s));")


@pytest.mark.parametrize("name,arrivals", [("prefill.cu", 4), ("skinny.cu", 1), ("attention.cu", 1)])
def test_slots_are_given_back_behind_the_stores(name, arrivals):
    text = source(name)
    assert len(re.findall(r"mbar_arrive\((?:cempty\(|rawempty\(|taken\))", text)) == arrivals
    assert faults(text) == []


def test_no_read_only_loads_of_the_few_token_kernel():
    assert re.findall(r"__ldg|\bldg_stream_\w+|ld\.global\.nc|__restrict__", source("fp4_linear.cu")) == []
