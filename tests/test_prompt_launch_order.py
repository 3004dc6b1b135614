"""The order of tensor memory and dependent launches in the kernels' sources, without a GPU.

A CTA of the next launch allocates its tensor memory before it waits for this launch to end.  If it could
come while a CTA of this launch still waits for columns, the two could wait for each other, and neither
wait has a limit.  So a kernel that allocates lets the next launch in only behind the allocation."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rope_block_sparse_b200", "csrc")


def code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def kernels(text):
    """Bodies of the __global__ functions."""
    for m in re.finditer(r"__global__", text):
        at = text.index("{", m.end())
        depth, end = 1, at + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        yield text[at:end]


LETS_IN = r"let_next_start\(|early_start\(|griddepcontrol\.launch_dependents"
ALLOCATING = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and "launch_early(" in code(f) and "tmem_alloc(" in code(f)]


def test_a_kernel_of_this_kind_is_found():
    assert ALLOCATING


@pytest.mark.parametrize("name", ALLOCATING)
def test_next_launch_comes_behind_the_allocation(name):
    text = code(name)
    inside = [k for k in kernels(text) if re.search(LETS_IN, k)]
    assert len(re.findall(LETS_IN, text)) == sum(len(re.findall(LETS_IN, k)) for k in inside)  # none in a function they call
    for body in inside:
        found = [m.start() for m in re.finditer(LETS_IN, body)]
        assert len(found) == 1
        branch = body[body.rindex("{", 0, found[0]):found[0]]  # the same warp's straight line of code
        assert "tmem_alloc(" in branch
