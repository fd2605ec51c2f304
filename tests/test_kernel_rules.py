"""Rules of the kernels' sources that no run shows reliably: they concern waits
that give up and blocks that start at different times (CPU only)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "learned_bit_lut_b200", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))


def code(path):
    """The source without its comments."""
    return re.sub(r"//[^\n]*", "", open(path).read())


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_warps_that_share_a_barrier_leave_together(path):
    """Behind a barrier of some warps, none decides by a flag that other warps
    may set meanwhile: a warp that leaves alone keeps the next barrier waiting."""
    assert not re.search(r"_sync\(\);\s*if \(\*abort(_flag)?\)", code(path))
