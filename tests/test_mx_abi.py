"""MXFP4 entry points on the CPU: refusals before any CUDA call, and pins of the tests' own
reference (hand-derived words, ties, ends of the range)."""
import ctypes

import numpy as np
import pytest

import decode_w4a16_g128_b200 as w4
import mx_reference as ref

lib = w4.lib
P = ctypes.c_void_p
A = 0x10000          # never dereferenced: validation fails first
B, C, D, E, F = (A + i * 0x1000000 for i in range(1, 6))


def quantize(w=A, dt=0, wq=B, s=C, N=4, K=64):
    return lib.w4a16_mx_quantize(P(w), dt, P(wq), P(s), N, K, P(0))


def dequantize(wq=B, s=C, w=A, dt=0, N=4, K=64):
    return lib.w4a16_mx_dequantize(P(wq), P(s), P(w), dt, N, K, P(0))


def matmul(x=A, wq=B, s=C, y=D, M=2, N=8, K=64):
    return lib.w4a16_mx_matmul(P(x), P(wq), P(s), P(y), M, N, K, P(0))


def matmul_a4(xq=A, xs=E, wq=B, s=C, y=D, M=2, N=8, K=64):
    return lib.w4a16_mx_matmul_a4(P(xq), P(xs), P(wq), P(s), P(y), M, N, K, P(0))


def gate_up(x=A, wq=B, s=C, h=D, M=2, N=8, K=64):
    return lib.w4a16_mx_gate_up(P(x), P(wq), P(s), P(h), M, N, K, P(0))


def backward(dy=A, wq=B, s=C, dx=D, M=2, N=8, K=64):
    return lib.w4a16_mx_matmul_backward(P(dy), P(wq), P(s), P(dx), M, N, K, P(0))


def gate_up_backward(x=A, wq=B, s=C, dh=D, dgu=E, dx=F, M=2, N=8, K=64):
    return lib.w4a16_mx_gate_up_backward(P(x), P(wq), P(s), P(dh), P(dgu), P(dx), M, N, K, P(0))


PRODUCTS = [matmul, matmul_a4, gate_up, backward, gate_up_backward]


@pytest.mark.parametrize("call", PRODUCTS)
def test_sizes(call):
    assert call(M=-1) == w4.ERR_INVALID_ARG
    assert call(N=-8) == w4.ERR_INVALID_ARG
    assert call(K=-32) == w4.ERR_INVALID_ARG
    assert call(K=48) == w4.ERR_UNSUPPORTED
    assert call(M=2 ** 31) == w4.ERR_UNSUPPORTED
    assert call(N=2 ** 31) == w4.ERR_UNSUPPORTED
    assert call(K=2 ** 31) == w4.ERR_UNSUPPORTED
    assert call(M=0) == w4.OK


@pytest.mark.parametrize("call", [quantize, dequantize])
def test_conversion_refusals(call):
    assert call(N=-1) == w4.ERR_INVALID_ARG
    assert call(K=-32) == w4.ERR_INVALID_ARG
    assert call(K=33) == w4.ERR_UNSUPPORTED
    assert call(N=2 ** 31) == w4.ERR_UNSUPPORTED
    assert call(dt=2) == w4.ERR_INVALID_ARG
    assert call(N=0) == w4.OK
    assert call(K=0) == w4.OK
    for name in ("w", "wq", "s"):
        assert call(**{name: 0}) == w4.ERR_INVALID_ARG
    for name in ("w", "wq", "s"):
        assert call(**{name: A + 0x900008}) == w4.ERR_MISALIGNED
    assert call(w=B) == w4.ERR_INVALID_ARG
    assert call(w=C - 16) == w4.ERR_INVALID_ARG


@pytest.mark.parametrize("call,buffers,output", [
    (matmul, ("x", "wq", "s", "y"), "y"),
    (matmul_a4, ("xq", "xs", "wq", "s", "y"), "y"),
    (gate_up, ("x", "wq", "s", "h"), "h"),
    (backward, ("dy", "wq", "s", "dx"), "dx"),
    (gate_up_backward, ("x", "wq", "s", "dh", "dgu", "dx"), "dx"),
    (gate_up_backward, ("x", "wq", "s", "dh", "dgu", "dx"), "dgu"),
])
def test_buffers(call, buffers, output):
    for b in buffers:
        assert call(**{b: 0}) == w4.ERR_INVALID_ARG, b
        assert call(**{b: A + 0x9000008}) == w4.ERR_MISALIGNED, b
    at = dict(zip(buffers, (A, B, C, D, E, F)))
    for b in buffers:
        if b != output:
            assert call(**dict(at, **{output: at[b]})) == w4.ERR_INVALID_ARG, b


@pytest.mark.parametrize("call", [gate_up, backward, gate_up_backward])
def test_rows_in_blocks_of_eight(call):
    assert call(N=12) == w4.ERR_UNSUPPORTED


def test_gate_up_row_limit():
    assert gate_up(N=2 ** 30) == w4.ERR_UNSUPPORTED
    assert gate_up_backward(N=2 ** 30) == w4.ERR_UNSUPPORTED


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    wq, s = torch.zeros(8, 8, dtype=torch.int32), torch.zeros(8, 2, dtype=torch.uint8)
    for call in (lambda: w4.w4a16_mx_quantize(x), lambda: w4.w4a16_mx_dequantize(wq, s),
                 lambda: w4.w4a16_mx_matmul(x, wq, s), lambda: w4.w4a16_mx_matmul_a4(wq, s, wq, s),
                 lambda: w4.w4a16_mx_gate_up(x, wq, s), lambda: w4.w4a16_mx_matmul_backward(x, wq, s),
                 lambda: w4.w4a16_mx_gate_up_backward(x, wq, s, x)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ pins of the reference


def test_reference_grid_and_packing():
    # words by hand: code k at bits 4k; 0x76543210 holds 0..7, 0xFEDCBA98 their negatives
    wq = np.array([[0x76543210, 0xFEDCBA98, 0, 0]], np.uint32)
    v = ref.values(wq, np.array([[128]], np.uint8))[0]
    assert v[:8].tolist() == [0, 1, 2, 3, 4, 6, 8, 12]
    assert v[8:16].tolist() == [0, -1, -2, -3, -4, -6, -8, -12]
    assert np.isnan(ref.values(wq, np.array([[255]], np.uint8))).all()


def test_reference_quantize_ties_and_ends():
    w = np.zeros((6, 32))
    w[0, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]        # ties go to the even codes
    w[1, :3] = [7.99, -0.2, -7.0]                                   # top in [4, 8): above 6 becomes 6
    w[2, 0] = 2.0 ** -149                                           # below every scale: e = 0
    w[3, :2] = [2.0 ** -126, -(2.0 ** -127)]
    w[4, 5] = np.inf
    w[5, :2] = [np.float64(np.finfo(np.float32).max), 1.0]
    wq, s = ref.quantize(w)
    v = ref.values(wq, s)
    assert s[:, 0].tolist() == [127, 127, 0, 0, 255, 252]
    assert v[0, :8].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]
    assert v[1, :3].tolist() == [6, 0, -6] and wq[1, 0] & 0xF0 == 0x80   # the zero keeps its sign
    assert v[2, 0] == 0 and v[3, :2].tolist() == [2.0 ** -126, -(2.0 ** -127)]
    assert np.isnan(v[4]).all() and not wq[4].any()
    assert v[5, 0] == 6 * 2.0 ** 125


def test_reference_bf16():
    assert ref.bf16(1 + 2.0 ** -8) == 1 and ref.bf16(1 + 3 * 2.0 ** -8) == 1 + 2.0 ** -6
    assert ref.bf16(2.0 ** -133) == 2.0 ** -133 and ref.bf16(2.0 ** -135) == 0
    assert ref.bf16(3.4e38) == np.inf and ref.bf16(-2.0) == -2.0


def test_reference_gradient_against_differences():
    rng = np.random.default_rng(1)
    w = ref.values(*ref.random_stored(rng, 32, 64, 122, 126))
    x, dh = rng.standard_normal((3, 64)), rng.standard_normal((3, 16))
    dgu, _ = ref.gate_up_backward(x, w, dh)
    dx = dgu @ w
    eps = 1e-6
    for m, k in ((0, 0), (1, 33), (2, 63)):
        e = np.zeros_like(x)
        e[m, k] = eps
        num = ((ref.gate_up(x + e, w)[0] - ref.gate_up(x - e, w)[0]) * dh).sum() / (2 * eps)
        # central differences: third derivative times eps^2 / 6 and rounding 2^-52 / eps of the sums
        assert abs(num - dx[m, k]) <= 1e-7 * (1 + np.abs(dgu[m]) @ np.abs(w[:, k]))
