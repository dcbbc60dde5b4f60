"""Products on both sides of the limits between the row kernel and the tensor-core kernels (rows of x,
size of the weight, length of a row): whole numbers, equal bit for bit; nothing outside the output is
written."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import decode_w4a16_g128_b200 as w4  # noqa: E402
import mx_reference as ref  # noqa: E402


def whole(rng, rows, k):
    x = torch.from_numpy(rng.integers(-8, 9, (rows, k)).astype(np.float32)).cuda()
    return x.bfloat16(), x.double()


def stored(rng, rows, k):
    wq, s = ref.random_stored(rng, rows, k, 126, 128)
    wq, s = torch.from_numpy(wq.view(np.int32).copy()).cuda(), torch.from_numpy(s.copy()).cuda()
    return wq, s, w4.w4a16_mx_dequantize(wq, s, dtype=torch.float32).double()


# sums are multiples of 1/4 below 96 K <= 2^22: exact in FP32
@pytest.mark.parametrize("M", [8, 9, 12, 16, 17, 32, 33])
@pytest.mark.parametrize("N,K", [(19664, 2560), (19456, 2560), (151, 12256), (151, 12288), (40, 16384), (33, 32768),
                                 (4736, 4096), (4737, 4096), (1000, 4128),
                                 (4737, 4128), (9456, 4128)])
def test_products_on_both_sides(M, N, K):
    rng = np.random.default_rng([50, M, N, K])
    wq, s, w = stored(rng, N, K)
    x, xd = whole(rng, M, K)
    buf = torch.full(((M + 16) * N // 8 * 8 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    lo = 8 * N
    y = w4.w4a16_mx_matmul(x, wq, s, buf[lo:lo + M * N].view(M, N))
    want = (xd @ w.T).float().bfloat16()
    assert torch.equal(y, want)
    assert (buf[:lo] == 7).all() and (buf[lo + M * N:] == 7).all()


@pytest.mark.parametrize("M", [1, 8, 9])
@pytest.mark.parametrize("N,K", [(4736, 1568), (4737, 1536), (4737, 1568), (9728, 2560), (33, 32768), (151, 9728)])
def test_4_bit_products_on_both_sides(M, N, K):
    rng = np.random.default_rng([51, M, N, K])
    wq, s, w = stored(rng, N, K)
    xq, xs, x = stored(rng, M, K)
    xs -= 3
    x = x / 8
    # products are multiples of 1/128, and no sum of them, in whatever order, reaches 2^24 of these
    assert float((x.abs() @ w.abs().T).max()) * 128 < 2 ** 24
    want = (x @ w.T).float().bfloat16()
    assert torch.equal(w4.w4a16_mx_matmul_a4(xq, xs, wq, s), want)


def test_long_rows_of_4_bit_values_on_the_tensor_cores():
    """Rows of 2^27 values, more of them than the row kernel takes: codes at a few places, zeros between."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    M, N, K = 9, 4, 2 ** 27
    rng = np.random.default_rng(52)
    at = [0, 39, K // 2 + 8, K - 40, K - 1]
    px, pw = rng.integers(0, 16, (M, len(at))), rng.integers(0, 16, (N, len(at)))

    def spread(picked):
        wq = torch.zeros(picked.shape[0], K // 8, dtype=torch.int32, device="cuda")
        nibbles = picked.astype(np.uint32) << np.array([4 * (i % 8) for i in at], np.uint32)
        wq[:, [i // 8 for i in at]] = torch.from_numpy(nibbles.view(np.int32)).cuda()
        return wq, torch.full((picked.shape[0], K // 32), 127, dtype=torch.uint8, device="cuda")

    y = w4.w4a16_mx_matmul_a4(*spread(px), *spread(pw)).double().cpu().numpy()
    assert np.array_equal(y, ref.bf16(ref.GRID[px] @ ref.GRID[pw].T))
    assert w4.w4a16_device_status() == w4.OK
