"""Where the gradient kernels put their sums by distance: the index arithmetic of a step, on the CPU."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "topology_scheduled_gb300", "csrc")


def _constants():
    """The integer constants that the kernels' index arithmetic is made of, as the sources define them."""
    text = "".join(open(os.path.join(SRC, f)).read() for f in ("score_terms.cuh", "backward_kernels.cuh"))
    found = {}
    for name, value in re.findall(r"constexpr int (k\w+) = ([^;]+);", text):
        if re.fullmatch(r"[\w\s+*()]+", value):
            try:
                found.setdefault(name, eval(value, {}, found))
            except NameError:
                pass
    return found


def test_sums_by_distance_stay_with_their_warp():
    """A near step adds to near_sums[d_lo + 32 - col0 + lane] and to the one 32 on, for every lane."""
    c = _constants()
    first, past = -c["kDistFront"], c["kNearRow"] - c["kDistFront"]
    assert past > c["kNearSums"]
    seen = set()
    for blocks in range(8):  # from the diagonal on
        for quarter in range(4):
            d_lo = blocks * c["kBlock"] + quarter * 32 - 63
            if d_lo + c["kWindow"] - 2 >= c["kNearSums"]:
                continue
            for col0 in (0, 32):
                for lane in range(32):
                    at = d_lo + 32 - col0 + lane
                    seen.update((at, at + 32))
    assert first <= min(seen) and max(seen) < past
    assert set(range(c["kNearSums"])) <= seen
