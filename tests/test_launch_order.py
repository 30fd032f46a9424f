"""Early dependent launches and tensor memory, by reading the kernels' sources (no GPU).

A grid that has signalled its dependents may share its SMs with them.  A kernel that takes tensor memory must
hold it before it signals, in every thread: a dependent that takes the columns first would wait for this grid to
end, and this grid for the columns."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_routed_expert_gb300", "csrc")
SOURCES = [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "tcgen05.alloc" in open(p).read()]


def events(text):
    """The calls that matter here, in the order of the source, comments left out."""
    text = re.sub(r"//[^\n]*", "", text)
    names = {"tcgen05.alloc": "alloc", "__syncthreads();": "sync", "pdl_launch_dependents();": "signal", "__global__": "kernel"}
    return [names[m.group(0)] for m in re.finditer("|".join(re.escape(n) for n in names), text)]


def test_some_kernels_take_tensor_memory():
    assert SOURCES


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_dependents_start_after_the_allocation(path):
    kernels = " ".join(events(open(path).read())).split("kernel")
    for k in (k.split() for k in kernels if "alloc" in k):
        signals = [i for i, e in enumerate(k) if e == "signal"]
        at = k.index("alloc")
        assert all(i > at and "sync" in k[at:i] for i in signals), k
