"""Attention over shared prefixes: what can be seen without a GPU."""
import os
import re

import pytest


def source(name):
    from speculative_decoding_verify_gb300 import build as b
    return open(os.path.join(b.CSRC, name)).read()


@pytest.mark.parametrize("name", ["sdv_rope.cu", "sdv_draw.cu", "sdv_paged_shared.cu", "sdv_paged_attn.cu", "sdv_paged_wide.cuh"])
def test_kernels_wait_for_what_they_read(name):
    """Every kernel waits for the launches before it, or takes the ticket that the plan released, whatever the call's arguments are."""
    text = source(name)
    kernels = re.findall(r"\n__global__.*?\n}\n", text, re.S)
    assert kernels
    for k in kernels:
        first = next(line.strip() for line in k.split("\n") if "pdl_wait()" in line or "after_plan(" in line)
        assert re.fullmatch(r"(if constexpr \(MODE == PA_OWN\) after_plan\(.*\)|pdl_wait\(\));", first), first
