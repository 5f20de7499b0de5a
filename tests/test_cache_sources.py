"""What no run on a GPU is sure to show: kernels that are set up while the kernel before them still writes read their inputs
by ordinary loads."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "topology_scheduled_gb300", "csrc")


def test_early_kernels_read_by_ordinary_loads():
    early = []
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        text = re.sub(r"//.*", "", open(path).read())
        if "wait_for_predecessor()" in text:
            early.append(os.path.basename(path))
            # no read-only loads, and nothing that lets the compiler make some
            assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", text), path
    assert sorted(early) == ["paged_decode.cu", "rotary.cu"]
