"""Static rule of the CUDA sources (no GPU): a kernel that may be placed while what runs before it still writes (one that
waits with griddepcontrol.wait) does not read through the read-only path, whose data has to be constant for as long as
the kernel is there."""

import re

from test_source_rules_cpu import _sources


def test_no_read_only_loads_where_kernels_are_placed_early():
    early = []
    for name, text in _sources():
        if name == "common.cuh":
            continue        # the waits' own definitions
        # the weight updates' first kernel is launched in the ordinary way, after all that may write the gradient, which
        # it and the next one read through functions that stand before them
        first = re.split(r"muon_start_kernel\(", text)[0] if name == "muon.cu" else ""
        if "wait_previous()" in text or "after_previous()" in text:
            early.append(name)
            rest = text[len(first):]
            assert "__ldg" not in rest and "ld.global.nc" not in rest, name
    assert {"layer_norm.cu", "linear_ce.cu", "dropout.cu"} <= set(early)
