"""Programmatic dependent launches: what an earlier kernel wrote may be read only after
griddepcontrol.wait, so a kernel calls it first and without a condition.  A kernel that reads
before it may see a row number of another batch, and would read and write out of range: this is
checked in the source, not by a run."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantised_gemm_gb300", "csrc")


def kernels(name):
    """(name, body) of each kernel of a file."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\(", text):
        begin = text.index("{\n", m.end())
        yield m.group(1), text[begin:text.index("\n}\n", begin)]


@pytest.mark.parametrize("name", ["adapter.cu", "adapter_low.cu", "adapter_high.cu", "adapter_weight.cu", "layer_norm.cu"])
def test_a_kernel_waits_before_it_reads(name):
    found = list(kernels(name))
    assert found
    for kernel, body in found:
        at = body.index("griddep_wait();")
        line = body[body.rindex("\n", 0, at) + 1:at]
        assert line == "  ", (kernel, line)  # a statement of the kernel's own, under no condition
        before = body[:at]
        assert not re.search(r"__ld|find_tile|load_|copy|\*\w|\w\[(?!\])", re.sub(r"__shared__[^;]*;", "", before)), (kernel, before)
        assert body.index("griddep_launch_dependents();") > at


def test_no_wait_depends_on_the_launch():
    """What a launch two before wrote is no more visible without the wait than what the last one wrote."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            for line in f:
                assert not re.search(r"if \(!?[\w.]+\) griddep_wait\(\)", line), (name, line)
