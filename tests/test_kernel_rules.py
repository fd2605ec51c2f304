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


@pytest.mark.parametrize("path", [p for p in SOURCES if p.endswith(".cu")], ids=os.path.basename)
def test_blocks_of_a_cluster_have_started_before_they_are_written_to(path):
    """Shared memory of another block is there once that block has started, which
    only a cluster barrier tells: each kernel has one before its first store
    into another block or arrival at one."""
    text = code(path)
    cuts = [m.start() for m in re.finditer(r"__global__", text)] + [len(text)]
    for kernel in (text[a:b] for a, b in zip(cuts, cuts[1:])):
        remote = re.search(r"st\.shared::cluster|st_async_v4\(|mbar_arrive_leader\(", kernel)
        if remote is None:
            continue
        started = r"block_sync\(\);" if "block_sync = " in kernel else r"barrier\.cluster\.wait|cluster_sync(_init)?\(\);"
        assert re.search(started, kernel[:remote.start()]), kernel[:80]


def test_dequantization_reads_the_weight_behind_its_wait():
    """It starts before the kernel ahead of it has ended, and that one may be
    whatever wrote the weight."""
    text = code(os.path.join(CSRC, "pack_dequant.cu"))
    body = text[text.index("dequant_rows_kernel("):]
    assert body.index("griddepcontrol.wait") < re.search(r"ld_\w+\(|__ldg\(", body).start()


def test_bounded_waits_do_not_count_the_kernel_before():
    """A wait that begins while the kernel ahead still runs ends when that one
    has; only then may its bound start."""
    waits = code(os.path.join(CSRC, "tcgen05.cuh"))
    assert waits.count("> kTcWaitCycles") == waits.count("t0 = clock_after_kernel_ahead()") == 3
    restart = waits[waits.index("clock_after_kernel_ahead() {"):]
    assert restart.index("griddepcontrol.wait") < restart.index("clock64()")
    decode = code(os.path.join(CSRC, "linear.cu"))
    producer = decode.index("if (warp == NW) {")
    assert decode.index("griddepcontrol.wait", producer) < decode.index("wait_bar(", producer)
