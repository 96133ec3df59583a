"""How the kernels launched by programmatic dependent launch read global memory.

Such a kernel is live while the kernel before it still writes.  A load through the
non-coherent path (`__ldg`, `ld.global.nc`, or a const __restrict__ pointer, which lets the
compiler choose it) asks for bytes that nobody writes during the kernel's whole life and is
not ordered by the wait for the previous kernel, so none may be in their sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_fp8_sm_gb300", "csrc")
SOURCES = ["block128_rows.cuh", "block128_tile.cuh", "block128_native.cuh", "quant_tokens.cuh", "block128_api.cu"]


def _code(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", SOURCES)
def test_no_noncoherent_load(name):
    found = re.findall(r"__ldg\w*|ld\.global\.nc\S*|__restrict__", _code(name))
    assert not found, f"{name}: {found}"


def test_every_kernel_waits_before_it_reads():
    """Each kernel of these files calls wait_for_previous before its first use of an operand."""
    for name, args in (("block128_rows.cuh", "a"), ("block128_tile.cuh", "a"), ("block128_native.cuh", "a"),
                       ("quant_tokens.cuh", "a")):
        for body in re.split(r"__global__", _code(name))[1:]:
            before = body[:body.index("wait_for_previous();")]
            uses = re.findall(rf"\b{args}\.(A|sA|B|sB|C|offsets|x|rows|q|s)\b", before)
            assert not uses, f"{name}: {uses}"
