"""The DRAM traffic that the benchmark reports belongs to the row-statistics kernel as it is: a change
of that kernel or of what it calls voids the figure, a change elsewhere in the same headers does not."""
import os
import shutil

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "speculative_decoding_verification_31_gb300", "csrc")


@pytest.fixture
def copy(tmp_path):
    for name in {s[0] for s in bench.ROW_STATS_SOURCES}:
        shutil.copy(os.path.join(CSRC, name), tmp_path)
    return tmp_path


def edit(path, old, new):
    text = path.read_text()
    assert text.count(old) >= 1
    path.write_text(text.replace(old, new, 1))


def test_the_figure_is_of_the_present_kernel():
    """(None: not captured since the kernel changed, and reported as null)"""
    assert bench.NCU_TRAFFIC["sources_sha1"] in (None, bench.kernel_sources_sha1())


def test_other_helpers_do_not_void_it(copy):
    edit(copy / "device_common.cuh", "namespace specverify {", "namespace specverify {\nconstexpr int kUnrelated = 1;\n")
    edit(copy / "device_common.cuh", "add.rn.f32x2", "add.f32x2")
    edit(copy / "kernels.cuh", "scan_greedy_kernel", "scan_greedy_renamed")
    assert bench.kernel_sources_sha1(str(copy)) == bench.kernel_sources_sha1()


@pytest.mark.parametrize("name,text", [("device_common.cuh", "ld.global.nc.L1::no_allocate.v4.u32"),
                                       ("device_common.cuh", "struct SoftmaxStat {"),
                                       ("kernels.cuh", "stream_pdl_wait();")])
def test_its_own_code_does(copy, name, text):
    edit(copy / name, text, text + " ")
    assert bench.kernel_sources_sha1(str(copy)) != bench.kernel_sources_sha1()
