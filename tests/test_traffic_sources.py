"""The committed DRAM traffic of the projections is void as soon as anything changes that decides it: kernels, work
split, tensor maps, or which kernel, grid and cluster a call launches."""
import os

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "weight_only_groupwise_gb300", "csrc")


def test_every_source_of_a_projection_counts():
    for f in os.listdir(CSRC):
        if f.endswith((".cu", ".cuh", ".h")):
            text = open(os.path.join(CSRC, f)).read()
            decides = any(w in text for w in ("proj_kernel", "encode_weight_maps", "launch_tc_proj", "make_plan"))
            assert not decides or f in bench.KERNEL_SOURCES, f


@pytest.mark.parametrize("name,line", [("nq_proj_tc.cu", "box"), ("nq_api.cu", "grid"), ("nq_proj_q4.cu", ";"), ("nq_tc.cuh", ";")])
def test_a_change_of_such_a_source_changes_the_hash(monkeypatch, tmp_path, name, line):
    before = bench.kernel_hash()
    folder = tmp_path / "weight_only_groupwise_gb300" / "csrc"
    folder.mkdir(parents=True)
    for f in os.listdir(CSRC):
        if f.endswith((".cu", ".cuh", ".h")):
            (folder / f).write_text(open(os.path.join(CSRC, f)).read())
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_hash() == before
    text = (folder / name).read_text()
    at = text.rindex(line)
    (folder / name).write_text(text[:at] + " + 1 " + text[at:])
    assert bench.kernel_hash() != before
    (folder / name).write_text("// a comment\n" + text)
    assert bench.kernel_hash() == before
    (folder / "nq_sample.cu").write_text("int other;")
    assert bench.kernel_hash() == before
