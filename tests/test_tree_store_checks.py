"""The debug build's claim that every global store's index is checked, for the kernels on drafted token
trees and the rows they write: each statement that stores, or forms the pointer it stores through,
stands behind an FA_IN_BOUNDS, in the statement or the few lines before it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "tiled_online_softmax_sm_gb300", "csrc")
# (pattern of the left side, how often)
STORES = {
    "tree_attn.cu": [(r"a\.cuts\[\w+\] = ", 2), (r"float4\* dst = a\.part_o \+", 1), (r"a\.part_s\[.*\] = ", 1),
                     (r"uint4\* dst = reinterpret_cast<uint4\*>\(a\.o \+", 1), (r"a\.lse\[.*\] =\s", 2),
                     (r"^\s*reinterpret_cast<uint2\*>\(a\.o \+", 1)],
    "tree_cache.cu": [(r"\bmask\[\w+\] = ", 1), (r"positions\[.*\] = ", 1), (r"base\[\(size_t\)to\[.*\] = ", 1),
                      (r"new_seq_lens\[\w+\] = ", 1), (r"^\s*to\[first.*\] = ", 1), (r"scale\[\(page0 \+ dst\).*\] = ", 1)],
    "qkv_rows.cu": [(r"\*reinterpret_cast<uint2\*>\(dst \+", 2)],
}


def _statements(name):
    """Lines without comments; a line that ends in `=` is joined with the next."""
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    return re.sub(r"=\n\s*", "= ", re.sub(r"//[^\n]*", "", text)).splitlines()


@pytest.mark.parametrize("name", sorted(STORES))
def test_stores_are_checked(name):
    lines = _statements(name)
    for pattern, times in STORES[name]:
        at = [i for i, line in enumerate(lines) if re.search(pattern, line)]
        assert len(at) == times, (pattern, [lines[i] for i in at])
        for i in at:
            assert any("FA_IN_BOUNDS" in x for x in lines[max(0, i - 9):i + 1]), lines[i]

