"""Calls on a stream that is given, while the current stream still works: memory that one of them uses is
not handed to the other.  The busy stream waits in a kernel that only counts clock cycles."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import decode_w4a16_g128_b200 as w4  # noqa: E402

M, N, K = 40, 512, 1024
BUSY = 20_000_000                      # clock cycles, some 10 ms


def calls():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    normal = lambda r, c: torch.randn(r, c, generator=g, device="cuda").bfloat16()
    x, dy, dh, w = normal(M, K), normal(M, N), normal(M, N // 2), normal(N, K)
    wq, s = w4.w4a16_mx_quantize(w)
    xq, xs = w4.w4a16_mx_quantize(x)
    layer = w4.w4a16_quantize(w)
    codes8 = torch.randint(-2 ** 31, 2 ** 31 - 1, (N, K // 4), generator=g, device="cuda", dtype=torch.int32)
    return {
        "affine quantize": (w4.w4a16_quantize, (w,)),
        "affine matmul": (w4.w4a16_matmul, (x, *layer)),
        "affine matmul_ex": (lambda *a, **kw: w4.w4a16_matmul_ex(*a, path=w4.PATH_GEMM, **kw), (x, *layer)),
        "affine last_rows": (lambda *a, **kw: w4.w4a16_matmul_last_rows(*a, 3, **kw), (x, *layer)),
        "affine gate_up": (w4.w4a16_gate_up, (x[:5], *layer)),
        "affine bits": (lambda *a, **kw: w4.w4a16_matmul_bits(*a, 8, **kw), (x[:20], codes8, *layer[1:])),
        "quantize": (w4.w4a16_mx_quantize, (x,)),
        "dequantize": (w4.w4a16_mx_dequantize, (wq, s)),
        "matmul": (w4.w4a16_mx_matmul, (x, wq, s)),
        "matmul_a4": (w4.w4a16_mx_matmul_a4, (xq, xs, wq, s)),
        "gate_up": (w4.w4a16_mx_gate_up, (x, wq, s)),
        "matmul_backward": (w4.w4a16_mx_matmul_backward, (dy, wq, s)),
        "gate_up_backward": (w4.w4a16_mx_gate_up_backward, (x, wq, s, dh)),
    }


NAMES = ["quantize", "dequantize", "matmul", "matmul_a4", "gate_up", "matmul_backward", "gate_up_backward",
         "affine quantize", "affine matmul", "affine matmul_ex", "affine last_rows", "affine gate_up", "affine bits"]


def every(name):
    call, args = calls()[name]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(*args)                                            # a first call, which may set a workspace up
    torch.cuda.synchronize()
    want = call(*args)
    torch.cuda.synchronize()
    return side, call, args, want if isinstance(want, tuple) else (want,)


def tuple_of(result):
    return result if isinstance(result, tuple) else (result,)


def equal(got, want):
    for a, b in zip(got, want):
        assert a.shape == b.shape and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_beside_pending_work_on_freed_memory(name, handle):
    side, call, args, want = every(name)
    victims = [torch.full_like(w, 3) for w in want]            # memory of the outputs' sizes
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    kept = [v.clone() for v in victims]                        # reads them once the busy kernel is over
    del victims
    got = tuple_of(call(*args, stream=side.cuda_stream if handle else side))
    side.synchronize()
    equal(got, want)
    torch.cuda.synchronize()
    assert all((k == 3).all() for k in kept)
    equal(got, want)                                           # nothing pending wrote over them


@pytest.mark.parametrize("name", NAMES)
def test_inputs_dropped_after_the_call(name):
    side, call, args, want = every(name)
    mine = [a.clone() for a in args]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = tuple_of(call(*mine, stream=side))
    shapes = [(a.shape, a.dtype) for a in mine]
    del mine
    others = [torch.ones(shape, dtype=dtype, device="cuda") for shape, dtype in shapes]
    torch.cuda.synchronize()
    equal(got, want)
    assert all((o == 1).all() for o in others)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_dropped_while_the_current_stream_reads_them(name):
    side, call, args, want = every(name)
    got = tuple_of(call(*args, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    kept = [t.clone() for t in got]
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(side):
        others = [torch.ones(shape, dtype=dtype, device="cuda") for shape, dtype in shapes]
    torch.cuda.synchronize()
    equal(kept, want)
    assert all((o == 1).all() for o in others)


@pytest.mark.parametrize("name", NAMES)
def test_the_default_stream_by_its_handle(name):
    """stream=0 from within another current stream: work in order with the default stream's."""
    side, call, args, want = every(name)
    torch.cuda._sleep(BUSY)                                    # on the default stream
    victims = [torch.full_like(w, 3) for w in want]
    with torch.cuda.stream(side):
        got = tuple_of(call(*args, stream=0))
    kept = [v.clone() for v in victims]
    torch.cuda.synchronize()
    equal(got, want)
    assert all((k == 3).all() for k in kept)
