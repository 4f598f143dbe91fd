"""The timing hook's kernel kinds (CPU). bench.py reports a kernel's measured traffic as long as the files it is built from, the
shared header among them, are those of the measurement: the kinds of other operators are listed elsewhere."""
import os
import re

import bench
from chunked_gated_delta_05_gb300 import _lib

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_gated_delta_05_gb300", "csrc")


def test_every_kind_has_a_name_of_its_own():
    L = _lib.load()
    names = [L.gdn_timing_name(k).decode() for k in range(L.gdn_timing_kinds())]
    assert len(set(names)) == len(names) and all(names)
    for name in (*bench.KERNEL_SOURCES, "tables", "conv_fwd", "norm_fwd", "norm_bwd", "conv_step", "delta_step", "sscan_fwd", "sscan_bwd", "sscan_step"):
        assert name in names, name
    assert L.gdn_timing_name(len(names)).decode() == ""


def test_the_shared_header_lists_no_other_operators_kinds():
    with open(os.path.join(CSRC, "common.cuh")) as f:
        shared = set(re.findall(r"\bkK[A-Z]\w*", f.read()))
    for name in ("block_api.cu",):
        with open(os.path.join(CSRC, name)) as f:
            used = set(re.findall(r"TimedScope \w+\((kK\w+)", f.read()))
        assert used and not used & shared, used & shared
