"""Sources of the kernels that may start before the kernel in front of them has ended (launch_dependent): what that one
writes is visible to ordinary loads behind wait_previous_kernel(), but not to loads through the read-only path, whose
data has to stay unchanged for as long as the kernel runs."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "route_kv_memory_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


FILES = sorted(n for n in os.listdir(CSRC) if n.endswith(".cu") and "launch_dependent(" in source(n))


def test_the_files_are_found():
    assert {"kv8.cu", "tc_attention.cu", "tc_attention_bwd.cu"} <= set(FILES)


@pytest.mark.parametrize("name", FILES)
def test_no_loads_through_the_read_only_path(name):
    text = source(name)
    assert not re.search(r"__ldg\s*\(|\bld\.global\.nc|__ldlu|__restrict__", text)


@pytest.mark.parametrize("name", FILES)
def test_every_dependent_kernel_waits(name):
    """Each kernel of these files that is launched as a dependent contains the wait (kv8.cu launches all of its own so)."""
    text = source(name)
    kernels = re.split(r"__global__", text)[1:]
    bodies = {re.search(r"(\w+_kernel)\s*\(", k).group(1): k for k in kernels}
    launched = set(bodies) if name == "kv8.cu" else set(re.findall(r"launch_dependent\(\s*(?:\w+::)*(\w+_kernel)", text))
    assert launched
    for k in launched:
        assert "wait_previous_kernel()" in bodies[k], k
