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


def test_no_kernel_is_built_that_no_call_reaches():
    """The kernel of few rows as compiled: whole sequences of 8 or 16 rows a group, rows behind a prefix the same but for 16 rows of D = 128 (the
    many-row kernel's), prefixes of D = 256 alone."""
    import shutil
    import subprocess
    from speculative_decoding_verify_gb300 import build as b
    b.build()
    obj = os.path.join(b.BUILD_DIR, "sdv_paged_attn.o")
    if not shutil.which("nm") or not os.path.exists(obj):
        pytest.skip("no list of the object's names")
    names = subprocess.run(["nm", obj], capture_output=True, text=True, check=True).stdout
    got = {tuple(int(x) for x in m) for m in re.findall(r"paged_attn_kernelILi(\d)ELi(\d+)ELi(\d)ELi(\d)EE", names)}
    want = {(t, d, nt, mode) for t in range(3) for d in (64, 128, 256) for nt in (1, 2) for mode in (0, 1) if (d, nt, mode) != (128, 2, 1)}
    assert got == want | {(t, 256, 2, 2) for t in range(3)}


def test_the_weights_unit_stands_in_one_place():
    """The join scales partials by the unit that the many-row kernel's weights are in."""
    names = ["sdv_paged_attn.cu", "sdv_paged_attn.cuh", "sdv_paged_wide.cuh", "sdv_paged_shared.cu"]
    assert sum(source(n).count("6.103515625e-05") for n in names) == 1
    assert "l.unit = PW_UNIT;" in source("sdv_paged_attn.cu")
