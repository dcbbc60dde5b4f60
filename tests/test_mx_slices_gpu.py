"""Rows cut out of stored weights and of quantised activations (a shard, the last tokens of a prompt):
scales that start at any address, in every function that reads them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import decode_w4a16_g128_b200 as w4  # noqa: E402
import mx_reference as ref  # noqa: E402


def dev(wq, s):
    return torch.from_numpy(wq.view(np.int32).copy()).cuda(), torch.from_numpy(s.copy()).cuda()


def same(got, want):
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("K", [96, 2880, 4064])
@pytest.mark.parametrize("M", [1, 20, 40, 150])
def test_cut_rows(M, K):
    """Equal, bit for bit, to the calls on copies of the same rows; captured too."""
    rng = np.random.default_rng([30, M, K])
    lo, N = 5, 48
    wq, s = dev(*ref.random_stored(rng, N + 9, K))
    xq, xs = dev(*ref.random_stored(rng, M + 4, K, 122, 128))
    cut = lambda t, a, n: t[a:a + n]
    w = cut(wq, lo, N), cut(s, lo, N)
    v = cut(xq, 3, M), cut(xs, 3, M)
    assert w[1].data_ptr() % 16 and v[1].data_ptr() % 16
    w2, v2 = tuple(t.clone() for t in w), tuple(t.clone() for t in v)
    x = torch.randn(M, K, device="cuda").bfloat16()
    dy, dh = torch.randn(M, N, device="cuda").bfloat16(), torch.randn(M, N // 2, device="cuda").bfloat16()

    def every(w, v):
        return [w4.w4a16_mx_dequantize(*w), w4.w4a16_mx_matmul(x, *w), w4.w4a16_mx_matmul_a4(*v, *w),
                w4.w4a16_mx_gate_up(x, *w), w4.w4a16_mx_matmul_backward(dy, *w),
                *w4.w4a16_mx_gate_up_backward(x, *w, dh)]

    want = every(w2, v2)
    for a, b in zip(every(w, v), want):
        same(a, b)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = w4.w4a16_mx_matmul(x, *w, stream=side)
    side.synchronize()
    same(y, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = every(w, v)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        same(a, b)


def test_cut_rows_against_the_formula():
    rng = np.random.default_rng(31)
    M, N, K = 40, 24, 96
    wq, s = ref.random_stored(rng, N + 1, K, 126, 128)
    x = rng.integers(-8, 9, (M, K)).astype(np.float64)
    xd = torch.from_numpy(x.astype(np.float32)).cuda().bfloat16()
    q, sd = (t[1:] for t in dev(wq, s))
    y = w4.w4a16_mx_matmul(xd, q, sd).double().cpu().numpy()
    assert np.array_equal(y, ref.bf16(x @ ref.values(wq, s)[1:].T))


def test_scales_to_be_written_have_to_be_aligned():
    w = torch.randn(4, 96, device="cuda")
    out = torch.full((8, 3), 7, dtype=torch.uint8, device="cuda")
    with pytest.raises(w4.W4A16Error) as e:
        w4.w4a16_mx_quantize(w, scales=out[1:5])
    assert e.value.status == w4.ERR_MISALIGNED and (out == 7).all()
