"""Kernels that are launched programmatically start before the kernel in front of them ends, so
their operands are not read-only for their whole life: they take no non-coherent loads (which the
compiler may also move above the wait)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_mixed_precision_mxq_b200", "csrc")


def source(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def test_programmatic_kernels_read_coherently():
    files = [p for p in glob.glob(os.path.join(CSRC, "*.cu")) if "grid_wait()" in source(p)]
    assert [os.path.basename(p) for p in files] == ["gemm_rows.cu"]
    for p in files:
        for what in ("__ldg", "ld.global.nc", "__restrict__"):
            assert what not in source(p), "%s in %s" % (what, os.path.basename(p))


def test_shared_headers_offer_them_no_such_load():
    for name in ("ptx.cuh", "mx_elem.cuh", "mxq_internal.h"):
        for what in ("__ldg", "ld.global.nc"):
            assert what not in source(os.path.join(CSRC, name)), "%s in %s" % (what, name)
