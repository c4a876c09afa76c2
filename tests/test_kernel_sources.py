"""What the sources of the chained kernels must not say (no GPU needed).

Kernels that let their successor start early (griddepcontrol.launch_dependents) are still writing when it starts.
A successor waits for them before it reads, but a pointer declared const and __restrict__ also tells the compiler
that nobody writes there during the kernel's whole life, and lets it read by the non-coherent path."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "kda_linear_attention_02_b200", "csrc")
# the kernels that start early behind one of those: theirs, and the decode kernels, launched the same way
CHAINED = sorted(glob.glob(os.path.join(CSRC, "kda_lin*.cu"))) + [os.path.join(CSRC, f) for f in ("kda_pages.cu", "kda_decode.cu")]


def kernels(text):
    """(name, parameters) of the __global__ functions."""
    for m in re.finditer(r"__global__", text):
        head = text[m.start():text.index("{", m.start())]
        head = re.sub(r"__launch_bounds__\((?:[^()]|\([^()]*\))*\)", "", head)
        name, args = re.search(r"(\w+)\s*\((.*)\)", head, re.S).groups()
        yield name, args


@pytest.mark.parametrize("path", CHAINED, ids=os.path.basename)
def test_chained_kernels_promise_no_constant_memory(path):
    text = re.sub(r"//[^\n]*", "", open(path).read())
    found = [(name, " ".join(a.split())) for name, args in kernels(text) for a in args.split(",")
             if re.search(r"\bconst\b[^*]*\*[^*]*__restrict__", a)]
    assert not found
    assert not re.search(r"__ldg\b|\.nc\b|\bld_once", text)


def test_early_starts_are_known():
    # a file that lets successors start early belongs to the list above
    early = [p for p in glob.glob(os.path.join(CSRC, "*.cu")) if "grid_launch_dependents" in open(p).read()]
    assert early and set(map(os.path.basename, early)) <= set(map(os.path.basename, CHAINED))
