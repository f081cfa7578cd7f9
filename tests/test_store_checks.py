"""The debug build's claim that every global store's index is checked, for the stores of partials:
each stands behind an FA_IN_BOUNDS of its index, within the statement or the few lines before it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "tiled_online_softmax_sm_gb300", "csrc")
# the statements that store partials, or form the pointer they are stored through
STORE = re.compile(r"\*reinterpret_cast<float4\*>\((a\.)?part_s \+|"
                   r"dst = reinterpret_cast<(float4|uint4)\*>\((a\.)?part_o \+|a\.pre\[\w+\] = ")


@pytest.mark.parametrize("name,stores", [("rows_e4m3.cu", 3), ("fwd_bf16_sm103.cuh", 2)])
def test_stores_of_partials_are_checked(name, stores):
    lines = open(os.path.join(CSRC, name), encoding="utf-8").read().splitlines()
    at = [i for i, line in enumerate(lines) if STORE.search(line)]
    assert len(at) == stores, [lines[i] for i in at]
    for i in at:
        assert any("FA_IN_BOUNDS" in x for x in lines[max(0, i - 6):i + 1]), lines[i]
