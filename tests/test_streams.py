"""Whose memory a new output is when a stream is given: fakes of torch's streams and of the C entry
points, on the CPU.  Memory of the current stream may have been freed there with work in front of it
still pending, which the given stream does not wait for."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import decode_w4a16_g128_b200 as w4  # noqa: E402


class Fake(torch.Tensor):
    """A host tensor that passes for one of device 0 and knows the stream of its memory."""
    owner = None

    @staticmethod
    def make(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype).as_subclass(Fake)

    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0

    def new_empty(self, shape, dtype=None):
        t = Fake.make(*shape, dtype=dtype or self.dtype)
        t.owner = Streams.current
        return t

    def record_stream(self, stream):
        Streams.recorded.append((self.data_ptr(), stream.cuda_stream))


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Streams:
    current, recorded, calls = 7, [], []


@pytest.fixture
def fake(monkeypatch):
    Streams.current, Streams.recorded, Streams.calls = 7, [], []

    @contextlib.contextmanager
    def use(stream):
        before, Streams.current = Streams.current, stream.cuda_stream
        yield
        Streams.current = before

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(Streams.current))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle or 99))   # 0: a new one
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: Streams.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    class Library:
        def __getattr__(self, name):
            def call(*args):
                stream = args[-2] if name == "w4a16_matmul_ex" else args[-1]
                Streams.calls.append((name, getattr(stream, "value", stream)))
                return 0
            call.__name__ = name
            return call

    monkeypatch.setattr(w4, "lib", Library())


def mx_calls(**kw):
    x, dy, dh = Fake.make(2, 64), Fake.make(2, 16), Fake.make(2, 8)
    wq, s = Fake.make(16, 8, dtype=torch.int32), Fake.make(16, 2, dtype=torch.uint8)
    xq, xs = Fake.make(2, 8, dtype=torch.int32), Fake.make(2, 2, dtype=torch.uint8)
    return {
        "quantize": ((x,), lambda: w4.w4a16_mx_quantize(x, **kw)),
        "dequantize": ((wq, s), lambda: w4.w4a16_mx_dequantize(wq, s, **kw)),
        "matmul": ((x, wq, s), lambda: w4.w4a16_mx_matmul(x, wq, s, **kw)),
        "matmul_a4": ((xq, xs, wq, s), lambda: w4.w4a16_mx_matmul_a4(xq, xs, wq, s, **kw)),
        "gate_up": ((x, wq, s), lambda: w4.w4a16_mx_gate_up(x, wq, s, **kw)),
        "matmul_backward": ((dy, wq, s), lambda: w4.w4a16_mx_matmul_backward(dy, wq, s, **kw)),
        "gate_up_backward": ((x, wq, s, dh), lambda: w4.w4a16_mx_gate_up_backward(x, wq, s, dh, **kw)),
    }


def affine_calls(**kw):
    x, w = Fake.make(2, 128), Fake.make(16, 128)
    wq, s, b = Fake.make(16, 16, dtype=torch.int32), Fake.make(16, 1), Fake.make(16, 1)
    wq8 = Fake.make(16, 32, dtype=torch.int32)
    return {
        "affine matmul": ((x, wq, s, b), lambda: w4.w4a16_matmul(x, wq, s, b, **kw)),
        "affine matmul_ex": ((x, wq, s, b), lambda: w4.w4a16_matmul_ex(x, wq, s, b, **kw)),
        "affine last_rows": ((x, wq, s, b), lambda: w4.w4a16_matmul_last_rows(x, wq, s, b, 1, **kw)),
        "affine gate_up": ((x, wq, s, b), lambda: w4.w4a16_gate_up(x, wq, s, b, **kw)),
        "affine bits": ((x, wq8, s, b), lambda: w4.w4a16_matmul_bits(x, wq8, s, b, 8, **kw)),
        "affine quantize": ((w,), lambda: w4.w4a16_quantize(w, **kw)),
    }


def calls(**kw):
    return {**mx_calls(**kw), **affine_calls(**kw)}


def outputs(result):
    return result if isinstance(result, tuple) else (result,)


@pytest.mark.parametrize("name", list(calls()))
@pytest.mark.parametrize("given", [Stream(9), 9], ids=["stream", "handle"])
def test_outputs_on_a_given_stream(fake, name, given):
    inputs, call = calls(stream=given)[name]
    for out in outputs(call()):
        assert out.owner == 9                                    # its memory is the given stream's
        assert (out.data_ptr(), 7) in Streams.recorded           # and the current stream may use it
    for t in inputs:                                             # which may be dropped after the call
        assert (t.data_ptr(), 9) in Streams.recorded
    assert [stream for _, stream in Streams.calls] == [9] and Streams.current == 7


@pytest.mark.parametrize("name", list(calls()))
@pytest.mark.parametrize("given", [None, Stream(7), 7], ids=["none", "stream", "handle"])
def test_outputs_on_the_current_stream(fake, name, given):
    _, call = calls(stream=given)[name]
    assert all(out.owner == 7 for out in outputs(call()))
    assert not Streams.recorded and [stream for _, stream in Streams.calls] == [7]


@pytest.mark.parametrize("name", list(calls()))
@pytest.mark.parametrize("given", [0, 1])
def test_outputs_on_the_default_stream_by_its_handle(fake, name, given):
    inputs, call = calls(stream=given)[name]
    for out in outputs(call()):
        assert out.owner == 0 and (out.data_ptr(), 7) in Streams.recorded
    for t in inputs:
        assert (t.data_ptr(), 0) in Streams.recorded
    Streams.current, Streams.recorded = 0, []
    assert all(out.owner == 0 for out in outputs(call())) and not Streams.recorded
