"""Rows cut out of stored weights or quantised activations: their scales, K/32 bytes a row, seldom start
on 16 bytes, which the C functions need.  The fakes of test_streams.py, on the CPU."""
import pytest

torch = pytest.importorskip("torch")

import decode_w4a16_g128_b200 as w4  # noqa: E402
from test_streams import Fake, Streams, Stream, fake  # noqa: E402,F401


@pytest.fixture
def library(fake, monkeypatch):  # noqa: F811
    class Library:
        got = []

        def __getattr__(self, name):
            def call(*args):
                Library.got.append(args)
                return 0
            call.__name__ = name
            return call

    monkeypatch.setattr(w4, "lib", Library())
    return Library.got


@pytest.mark.parametrize("given", [None, Stream(9)], ids=["current", "given"])
def test_scales_of_cut_rows_are_handed_over_aligned(library, given):
    whole, half = Fake.make(20, 2, dtype=torch.uint8), Fake.make(20, 2, dtype=torch.uint8)
    wq, s, xq, xs = Fake.make(16, 8, dtype=torch.int32), whole[3:19], Fake.make(2, 8, dtype=torch.int32), half[5:7]
    x, dy, dh = Fake.make(2, 64), Fake.make(2, 16), Fake.make(2, 8)
    assert s.data_ptr() % 16 and xs.data_ptr() % 16
    w4.w4a16_mx_dequantize(wq, s, stream=given)
    w4.w4a16_mx_matmul(x, wq, s, stream=given)
    w4.w4a16_mx_matmul_a4(xq, xs, wq, s, stream=given)
    w4.w4a16_mx_gate_up(x, wq, s, stream=given)
    w4.w4a16_mx_matmul_backward(dy, wq, s, stream=given)
    w4.w4a16_mx_gate_up_backward(x, wq, s, dh, stream=given)
    at = [library[0][1], library[1][2], library[2][1], library[2][3], library[3][2], library[4][2], library[5][2]]
    assert len(library) == 6 and all(a % 16 == 0 for a in at), at
    whole16 = Fake.make(40, 2, dtype=torch.uint8)[8:24]
    w4.w4a16_mx_matmul(x, wq, whole16)
    assert library[-1][2] == whole16.data_ptr()              # aligned ones are not copied
