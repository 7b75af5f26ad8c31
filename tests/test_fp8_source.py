"""What the 8-bit products must have in their source and no run can show for certain. No GPU."""
import os
import re

import pytest

from tests.test_step_source import CSRC, body

KERNELS = ["fp8_rows_kernel", "fp8_cols_kernel"]


def role(text: str, begin: str, end: str) -> str:
    """A warp's part of a kernel."""
    at = text.index(begin)
    return text[at:text.index(end, at)]


@pytest.mark.parametrize("kernel", KERNELS)
def test_no_block_leaves_while_its_copies_are_on_their_way(kernel):
    """Any warp can give up waiting, also after the producer has asked for its last copies: it waits for them in any case."""
    producer = role(body("nq_fp8.cuh", kernel), "if (warp == kProducer)", "else if (warp == kMma)")
    tail = producer[producer.rindex("f8_gather4("):]
    drain = re.search(r"for \(int j = seq > kStages \? seq - kStages : 0; j < seq; \+\+j\)\s*mbar_wait_drain\(full0", tail)
    assert drain
    # a statement of its own, behind the one for an aborted call's first rows
    assert tail[:drain.start()].rstrip().endswith("__syncwarp();") and "x_late(seq);" in tail[:drain.start()]
    assert not re.search(r"(if|else|while|for)\s*(\([^;{}]*\))?\s*$", tail[:drain.start()].rstrip())
    assert tail.count("mbar_wait_drain") == 1


@pytest.mark.parametrize("kernel", KERNELS)
def test_bounded_waits_begin_when_the_call_ahead_has_ended(kernel):
    """Every warp of a dense call: waits count their own time alone. The producer's first turn through its stages needs no wait,
    and ends with the rows of x, which it asks for when the call ahead has ended."""
    text = body("nq_fp8.cuh", kernel)
    mma = role(text, "else if (warp == kMma)", "else if (warp == kScales)")
    assert mma.index("grid_dependency_wait();") < mma.index("mbar_wait(")
    epilogue = role(text, "regs_more<", "tmem_dealloc")
    assert epilogue.index("grid_dependency_wait();") < epilogue.index("mbar_wait(")
    producer = role(text, "if (warp == kProducer)", "else if (warp == kMma)")
    late = role(producer, "auto x_late", "};")
    assert late.index("grid_dependency_wait();") < late.index("f8_copy_2d(")
    assert "if (seq + 1 == late) x_late(late);" in producer


def test_resident_clusters_are_counted_on_each_device():
    """What is asked of the driver once is asked for the device that is current, as devices differ; a failure on one stays there."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "nq_fp8.cu")).read())
    at = text.index("fp8_clusters(int ")
    f = text[at:text.index("\n}\n", at)]
    assert re.match(r"fp8_clusters\(int dev, int sms\)", f)
    assert "static std::once_flag once[kDevices];" in f and "static int most[kDevices][kF8MostSplit + 1]" in f
    assert "std::call_once(once[dev]," in f and "most[dev]" in f
    assert re.search(r"dev < 0 \|\| dev >= kDevices", f)
    assert re.findall(r"fp8_clusters\(([^)]*)\)", text)[1:] == ["dev, d.sms"]
