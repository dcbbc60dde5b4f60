"""What orders the affine GEMM's accesses and no result shows: looks at the sources, on the CPU.

The tensor-core layer and its preparation kernel begin before the preceding kernel of the stream has
ended.  What the library's own kernels write right before them (x, from the layer in front; the bias
step's coefficients) must not be read through the non-coherent path, whose data may not change during a
kernel."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_w4a16_g128_b200", "csrc")
GEMM = os.path.join(CSRC, "gemm.cuh")


def test_fresh_data_by_plain_loads():
    text = re.sub(r"//[^\n]*", "", open(GEMM).read())
    assert "ldg_nc" not in text and ".global.nc" not in text
    loads = re.findall(r"__ldg\(([^;]*)\)", text)
    assert all(re.match(r"(biases|scales|src) \+", a) for a in loads), loads    # the weights' parameters alone
    assert not re.search(r"__restrict__ x\b", text)


def test_a_warp_gives_up_as_one():
    """A limited wait whose outcome decides where a whole warp goes on has one outcome for the warp: lanes
    that left at different times would miss collective instructions."""
    text = open(GEMM).read()
    roles = text[text.index("--- dequantisation (both CTAs)"):]
    assert roles.count("!mbar_wait_warp(") == 5 and "mbar_wait(" not in roles
