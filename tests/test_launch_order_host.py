"""Kernels that may start before what is in front of them has ended read nothing of it
before they wait for it. (A missing wait shows on a GPU by chance only, so the order is
read from the sources.)"""
import os
import re

import pytest

import paged_kv_varlen_attn_gb300 as pa

CSRC = os.path.join(os.path.dirname(pa.__file__), "csrc")
READS = re.compile(r"\bi4_seq\(|\bi4_start\(|__ldg\(|__ldcg\(|tma_load_\dd\(|a\.(cu|seqused_k|bt|table"
                   r"|sinks|q)\[")


def body(source, kernel):
    """The text of a kernel's definition, without comments."""
    text = open(os.path.join(CSRC, source)).read()
    text = re.sub(r"//[^\n]*", "", text)
    at = text.index(kernel + "(const __grid_constant__")
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]
    raise AssertionError(kernel)


@pytest.mark.parametrize("source,kernel", [("int4_decode.cu", "int4_decode_kernel"),
                                           ("int4_decode.cu", "int4_combine_kernel")])
def test_waits_before_it_reads(source, kernel):
    text = body(source, kernel)
    wait = text.index("pdl_wait()")
    first = READS.search(text)
    assert first and wait < first.start(), text[first.start():first.start() + 60]
    # No way out in front of the wait: the grid ends after its predecessor.
    assert "return" not in text[:wait]
