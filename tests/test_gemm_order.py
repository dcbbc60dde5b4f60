"""The tensor-core layer and its preparation kernel begin before the preceding kernel of the stream has
ended.  What the library's own kernels write right before them (x, from the layer in front; the bias
step's coefficients) must not be read through the non-coherent path, whose data may not change during a
kernel: a look at the source, on the CPU."""
import os
import re

GEMM = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_w4a16_g128_b200", "csrc",
                    "gemm.cuh")


def test_fresh_data_by_plain_loads():
    text = re.sub(r"//[^\n]*", "", open(GEMM).read())
    assert "ldg_nc" not in text and ".global.nc" not in text
    loads = re.findall(r"__ldg\(([^;]*)\)", text)
    assert all(re.match(r"(biases|scales|src) \+", a) for a in loads), loads    # the weights' parameters alone
    assert not re.search(r"__restrict__ x\b", text)
