"""MXFP4 operators on the GPU against tests/mx_reference.py (64 bits, derived tolerances).

Exact problems (small whole x, scales that keep every sum a whole number of quarters below 2^24)
have to match bit for bit: a wrong index, block or row cannot hide in a tolerance."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import decode_w4a16_g128_b200 as w4  # noqa: E402
import mx_reference as ref  # noqa: E402


def dev_bf16(a):
    """Values exact in BF16 -> a bfloat16 CUDA tensor."""
    return torch.from_numpy(ref.bf16_bits(a).view(np.int16).copy()).cuda().view(torch.bfloat16).reshape(a.shape)


def dev(wq, s):
    return torch.from_numpy(wq.view(np.int32).copy()).cuda(), torch.from_numpy(s.copy()).cuda()


def host(t):
    return t.double().cpu().numpy()


def codes(wq, s):
    return wq.cpu().numpy().view(np.uint32), s.cpu().numpy()


def near(got, want, tol, what=""):
    d = np.abs(got - want)
    bad = ~(d <= tol) & ~(np.isnan(got) & np.isnan(want)) & ~((got == want) & np.isinf(got))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[:4].tolist()}: " \
        f"{got[bad][:4]} for {want[bad][:4]}, tolerance {np.broadcast_to(tol, got.shape)[bad][:4]}"


def same(got, want, what=""):
    bad = ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} differ, first at {np.argwhere(bad)[:6].tolist()}: " \
        f"{got[bad][:4]} for {want[bad][:4]}"


def normal(rng, rows, k, scale=1.0):
    """BF16 values, one in a hundred twenty times as large."""
    x = rng.standard_normal((rows, k)) * scale
    x[rng.random((rows, k)) < 0.01] *= 20
    return ref.bf16(x)


def whole(rng, rows, k):
    return rng.integers(-8, 9, (rows, k)).astype(np.float64)


# ------------------------------------------------------------------ quantiser


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,K", [(1, 32), (1, 2560), (3, 96), (7, 4064), (129, 160), (33, 32)])
def test_quantize(N, K, dtype):
    rng = np.random.default_rng([1, N, K])
    w = (rng.standard_normal((N, K)) * np.exp2(rng.integers(-30, 30, (N, 1)))).astype(np.float32)
    if dtype == "bf16":
        w = ref.bf16(w).astype(np.float32)
    t = torch.from_numpy(w).cuda()
    wq, s = w4.w4a16_mx_quantize(t if dtype == "f32" else t.bfloat16())
    rq, rs = ref.quantize(w)
    gq, gs = codes(wq, s)
    assert np.array_equal(gs, rs) and np.array_equal(gq, rq)
    for dt in (torch.bfloat16, torch.float32):
        same(host(w4.w4a16_mx_dequantize(wq, s, dtype=dt)), ref.values(rq, rs), "values")


def corner_rows():
    w = np.zeros((12, 64), np.float32)
    w[0, :16] = np.repeat([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 2) * np.tile([1, -1], 8)
    w[1, :4] = [7.99, -0.2, -7.0, -0.0]
    w[2, 0] = 2.0 ** -149
    w[3, :3] = [2.0 ** -126, -(2.0 ** -127), 2.0 ** -128]
    w[4, 5] = np.inf
    w[5, 40] = np.nan
    w[6, :2] = [np.finfo(np.float32).max, 1.0]
    w[7] = -0.0
    w[8] = np.float32(2.0 ** -125)
    w[9, 31], w[9, 32] = -np.inf, 3.0
    w[10] = np.linspace(-8, 8, 64)
    w[11] = np.nextafter(np.float32(2.5), np.float32(3)) * np.float32(2.0 ** -20)
    return w


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_corners(dtype):
    w = corner_rows()
    t = torch.from_numpy(w).cuda()
    if dtype == "bf16":
        w = host(t.bfloat16()).astype(np.float32)
        t = t.bfloat16()
    rq, rs = ref.quantize(w)
    wq, s = w4.w4a16_mx_quantize(t)
    gq, gs = codes(wq, s)
    assert np.array_equal(gs, rs) and np.array_equal(gq, rq)
    same(host(w4.w4a16_mx_dequantize(wq, s)), ref.values(rq, rs))


def test_dequantize_every_scale():
    """All 256 scale bytes with all 16 codes; beyond FP32's range the value is an infinity."""
    wq = np.tile(np.array([0x76543210, 0xFEDCBA98, 0x01234567, 0x89ABCDEF], np.uint32), (256, 1))
    s = np.arange(256, dtype=np.uint8)[:, None]
    want = ref.values(wq, s)
    with np.errstate(invalid="ignore"):
        want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    d = dev(wq, s)
    for dt in (torch.bfloat16, torch.float32):
        same(host(w4.w4a16_mx_dequantize(*d, dtype=dt)), want)


# ------------------------------------------------------------------ products

SIZES = [(1, 8, 32), (1, 1, 64), (1, 1000, 2560), (2, 17, 96), (3, 129, 128), (5, 64, 9728), (8, 255, 1056),
         (9, 40, 64), (16, 300, 544), (17, 96, 96), (31, 33, 2592), (32, 1024, 256), (33, 130, 160), (64, 257, 512),
         (77, 1001, 1056), (127, 128, 32), (128, 256, 2560), (129, 1000, 352), (257, 520, 224), (300, 72, 4064)]
EIGHTS = [(m, max(8, n // 8 * 8), k) for m, n, k in SIZES]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul(M, N, K):
    rng = np.random.default_rng([2, M, N, K])
    wq, s = ref.random_stored(rng, N, K)
    w, x = ref.values(wq, s), normal(rng, M, K)
    y, tol = ref.product(x, w)
    near(host(w4.w4a16_mx_matmul(dev_bf16(x), *dev(wq, s))), y, tol)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul_exact(M, N, K):
    rng = np.random.default_rng([3, M, N, K])
    wq, s = ref.random_stored(rng, N, K, 126, 128)      # multiples of 1/4 up to 12: sums below 2^22 / 4
    x = whole(rng, M, K)
    same(host(w4.w4a16_mx_matmul(dev_bf16(x), *dev(wq, s))), ref.bf16(x @ ref.values(wq, s).T))


@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul_a4_exact(M, N, K):
    rng = np.random.default_rng([4, M, N, K])
    wq, s = ref.random_stored(rng, N, K, 126, 128)
    xq, xs = ref.random_stored(rng, M, K, 127, 128)     # sums below 2^24 / 8
    y = ref.values(xq, xs) @ ref.values(wq, s).T
    same(host(w4.w4a16_mx_matmul_a4(*dev(xq, xs), *dev(wq, s))), ref.bf16(y))


@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul_a4(M, N, K):
    """The whole path: activations quantised on the way."""
    rng = np.random.default_rng([5, M, N, K])
    wq, s = ref.random_stored(rng, N, K)
    x = normal(rng, M, K)
    xq, xs = w4.w4a16_mx_quantize(dev_bf16(x))
    rq, rs = ref.quantize(x)
    assert np.array_equal(codes(xq, xs)[0], rq) and np.array_equal(codes(xq, xs)[1], rs)
    y, tol = ref.product(ref.values(rq, rs), ref.values(wq, s))
    near(host(w4.w4a16_mx_matmul_a4(xq, xs, *dev(wq, s))), y, tol)


@pytest.mark.parametrize("M,N,K", EIGHTS)
def test_gate_up(M, N, K):
    rng = np.random.default_rng([6, M, N, K])
    wq, s = ref.random_stored(rng, 2 * N, K)
    x = normal(rng, M, K, 0.3)
    h, tol = ref.gate_up(x, ref.values(wq, s))
    near(host(w4.w4a16_mx_gate_up(dev_bf16(x), *dev(wq, s))), h, tol)


def test_gate_up_is_the_two_layers():
    """Exact sums: the fused block against the two layers' own FP32 sums, both interleavings' rows."""
    rng = np.random.default_rng(7)
    M, N, K = 19, 48, 96
    gq, gs = ref.random_stored(rng, N, K, 122, 123)
    uq, us = ref.random_stored(rng, N, K, 122, 123)
    wq, s = ref.interleave(gq, uq), ref.interleave(gs, us)
    x = whole(rng, M, K)
    g, u = x @ ref.values(gq, gs).T, x @ ref.values(uq, us).T
    h = g * ref.sigmoid(g) * u
    got = host(w4.w4a16_mx_gate_up(dev_bf16(x), *dev(wq, s)))
    near(got, h, (ref.HALF_STEP + 2 * ref.scalar(g)) * np.abs(h) + ref.TINY)
    t = w4.interleave_gate_up(dev(gq, gs)[0], dev(uq, us)[0])
    assert np.array_equal(t.cpu().numpy().view(np.uint32), wq)


@pytest.mark.parametrize("M,N,K", EIGHTS)
def test_matmul_backward(M, N, K):
    rng = np.random.default_rng([8, M, N, K])
    wq, s = ref.random_stored(rng, N, K)
    dy = normal(rng, M, N, 0.01)
    dx, tol = ref.product(dy, ref.values(wq, s).T)
    near(host(w4.w4a16_mx_matmul_backward(dev_bf16(dy), *dev(wq, s))), dx, tol)


@pytest.mark.parametrize("M,N,K", EIGHTS)
def test_matmul_backward_exact(M, N, K):
    rng = np.random.default_rng([9, M, N, K])
    wq, s = ref.random_stored(rng, N, K, 126, 128)
    dy = whole(rng, M, N)
    same(host(w4.w4a16_mx_matmul_backward(dev_bf16(dy), *dev(wq, s))), ref.bf16(dy @ ref.values(wq, s)))


@pytest.mark.parametrize("M,N,K", EIGHTS)
def test_gate_up_backward(M, N, K):
    rng = np.random.default_rng([10, M, N, K])
    wq, s = ref.random_stored(rng, 2 * N, K)
    w = ref.values(wq, s)
    x, dh = normal(rng, M, K, 0.3), normal(rng, M, N, 0.1)
    dx, dgu = w4.w4a16_mx_gate_up_backward(dev_bf16(x), *dev(wq, s), dev_bf16(dh))
    want, tol = ref.gate_up_backward(x, w, dh)
    got = host(dgu)
    near(got, want, tol, "dgu")
    y, ytol = ref.product(got, w.T)                    # the second product, from the rounded dgu
    near(host(dx), y, ytol, "dx")
    near(host(dx), want @ w, tol @ np.abs(w) + ytol, "dx against the formula")


def test_gate_up_backward_against_differences():
    """dx against central differences of the 64-bit forward pass."""
    rng = np.random.default_rng(11)
    M, N, K = 4, 24, 64
    wq, s = ref.random_stored(rng, 2 * N, K, 121, 124)
    w = ref.values(wq, s)
    x, dh = ref.bf16(rng.standard_normal((M, K))), ref.bf16(rng.standard_normal((M, N)))
    dx = host(w4.w4a16_mx_gate_up_backward(dev_bf16(x), *dev(wq, s), dev_bf16(dh))[0])
    dgu, tol = ref.gate_up_backward(x, w, dh)
    bound = tol @ np.abs(w) + ref.HALF_STEP * (np.abs(dgu @ w) + tol @ np.abs(w)) + 1e-6
    eps = 1e-5
    num = np.zeros_like(x)
    for k in range(K):
        e = np.zeros_like(x)
        e[:, k] = eps
        num[:, k] = ((ref.gate_up(x + e, w)[0] - ref.gate_up(x - e, w)[0]) * dh).sum(1) / (2 * eps)
    near(dx, num, bound + (ref.sum_error(dgu, w.T)))


# Sizes at which the kernels take their other shapes: several rounds of tiles a CTA, every tile width,
# a contraction shared by up to eight CTAs or four pairs, single CTAs, rows that start at odd addresses.
# The reference is a product of whole numbers in 64 bits on the GPU.
LARGE = [(2048, 4104, 544), (257, 19456, 96), (640, 5001, 640), (129, 333, 9728), (128, 19456, 256), (64, 4096, 2560),
         (100, 151, 8192), (1000, 10007, 512), (2047, 2056, 1312), (512, 1000, 9728), (40, 2560, 9728), (300, 9728, 160),
         (40, 1280, 4096), (40, 640, 9728), (40, 1000, 16384), (40, 2048, 16384), (300, 1600, 4096), (300, 2048, 4096),
         (300, 4096, 2560), (40, 16384, 992), (64, 9728, 640),
         # whole rounds of tiles, then shared ones
         (64, 19456, 2560), (2048, 19456, 2560), (300, 2560, 9728), (64, 2560, 19456), (2048, 9728, 2560),
         # the widest tiles of outputs that start at odd addresses, alone and in pairs
         (40, 2047, 16384), (90, 18001, 2048), (2000, 4001, 2048)]


def whole_on_gpu(rng, rows, k):
    x = torch.from_numpy(rng.integers(-8, 9, (rows, k)).astype(np.float32)).cuda()
    return x.bfloat16(), x.double()


def values_on_gpu(wq, s):
    return w4.w4a16_mx_dequantize(wq, s, dtype=torch.float32).double()


def equal(got, want):
    bad = got != want.float().bfloat16()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[:4].tolist()}"


@pytest.mark.parametrize("M,N,K", LARGE)
def test_large_exact(M, N, K):
    rng = np.random.default_rng([20, M, N, K])
    wq, s = dev(*ref.random_stored(rng, N, K, 126, 128))
    w = values_on_gpu(wq, s)
    x, xd = whole_on_gpu(rng, M, K)
    y = xd @ w.T                                   # multiples of 1/4 below 2^22: exact in FP32 too
    equal(w4.w4a16_mx_matmul(x, wq, s), y)
    xq, xs = w4.w4a16_mx_quantize(x)               # whole numbers up to 8: blocks of scale 1 or 2
    equal(w4.w4a16_mx_matmul_a4(xq, xs, wq, s), values_on_gpu(xq, xs) @ w.T)
    if N % 8 == 0:
        dy, dyd = whole_on_gpu(rng, M, N)
        equal(w4.w4a16_mx_matmul_backward(dy, wq, s), dyd @ w)
    assert w4.w4a16_device_status() == w4.OK


@pytest.mark.parametrize("M,N,K", [(2048, 2056, 544), (509, 9728, 256), (128, 9728, 256), (64, 1000, 2560), (17, 4864, 96),
                                   (64, 9728, 2560), (1024, 9728, 2560)])
def test_large_gated(M, N, K):
    rng = np.random.default_rng([21, M, N, K])
    wq, s = ref.random_stored(rng, 2 * N, K, 119, 121)
    wq, s = dev(wq, s)
    w = values_on_gpu(wq, s)
    x, xd = whole_on_gpu(rng, M, K)
    dh, dhd = whole_on_gpu(rng, M, N)
    gu = (xd @ w.T).reshape(M, -1, 2, 8)           # exact in FP32: multiples of 2^-9, below 2^9
    g, u = gu[:, :, 0], gu[:, :, 1]
    t = torch.sigmoid(g)
    scalar = (4 + 1.173 * g.abs()) * 2.0 ** -23 + 12 * 2.0 ** -24     # see mx_reference.scalar

    def close(got, want, err):
        bad = (got.double() - want).abs() > ref.HALF_STEP * (want.abs() + err) + err + ref.TINY
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[:4].tolist()}"

    h = g * t * u
    close(w4.w4a16_mx_gate_up(x, wq, s), h.reshape(M, N), (scalar * h.abs()).reshape(M, N))
    dx, dgu = w4.w4a16_mx_gate_up_backward(x, wq, s, dh)
    d = dhd.reshape(M, -1, 8)
    dg, du = d * u * t * (1 + g * (1 - t)), d * g * t
    eg = scalar * d.abs() * u.abs() * t * (1 + 2 * g.abs())
    close(dgu, torch.stack([dg, du], 2).reshape(M, 2 * N), torch.stack([eg, scalar * du.abs()], 2).reshape(M, 2 * N))
    want = dgu.double() @ w
    err = (2 * N / 16 + 32) * 2.0 ** -23 * (dgu.double().abs() @ w.abs())
    close(dx, want, err)
    assert w4.w4a16_device_status() == w4.OK


def test_first_call_of_a_process_captured():
    """No call needs a warm-up before it is captured, not even the first one on the device."""
    import os
    import subprocess
    import sys
    code = """
import torch, decode_w4a16_g128_b200 as w4
x = torch.ones(40, 64, dtype=torch.bfloat16, device="cuda")
w = torch.ones(32, 64, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    wq, s = w4.w4a16_mx_quantize(w)
    y = w4.w4a16_mx_matmul(x, wq, s)
    h = w4.w4a16_mx_gate_up(x, wq, s)
    y4 = w4.w4a16_mx_matmul_a4(*w4.w4a16_mx_quantize(x), wq, s)
    dx, dgu = w4.w4a16_mx_gate_up_backward(x, wq, s, h)
    v = w4.w4a16_mx_dequantize(wq, s)
g.replay()
torch.cuda.synchronize()
assert (y == 64).all() and (y4 == 64).all() and (h == 4096).all() and (v == 1).all(), (y, y4, h, v)
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "captured" in out.stdout, out.stdout + out.stderr


# ------------------------------------------------------------------ empty and odd calls


def test_empty():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    wq, s = torch.zeros(8, 8, dtype=torch.int32, device="cuda"), torch.zeros(8, 2, dtype=torch.uint8, device="cuda")
    assert w4.w4a16_mx_matmul(x, wq, s).shape == (0, 8)
    assert w4.w4a16_mx_matmul_backward(torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"), wq, s).shape == (0, 64)
    e = torch.empty(3, 0, dtype=torch.bfloat16, device="cuda")
    wq0, s0 = torch.empty(16, 0, dtype=torch.int32, device="cuda"), torch.empty(16, 0, dtype=torch.uint8, device="cuda")
    for y in (w4.w4a16_mx_matmul(e, wq0, s0), w4.w4a16_mx_gate_up(e, wq0, s0),
              w4.w4a16_mx_matmul_a4(wq0[:3], s0[:3], wq0, s0)):
        assert (y.view(torch.int16) == 0).all() and y.shape[0] == 3
    n0 = torch.empty(0, 8, dtype=torch.int32, device="cuda"), torch.empty(0, 2, dtype=torch.uint8, device="cuda")
    dx = w4.w4a16_mx_matmul_backward(e, *n0)
    assert dx.shape == (3, 64) and (dx.view(torch.int16) == 0).all()


@pytest.mark.parametrize("M", [1, 6, 20, 70, 140])
def test_rows_behind_the_last_stay(M):
    rng = np.random.default_rng(12)
    N, K = 136, 160
    wq, s = ref.random_stored(rng, N, K, 126, 128)
    d = dev(wq, s)
    x, dy = whole(rng, M, K), whole(rng, M, N)
    for width, call in ((N, lambda y: w4.w4a16_mx_matmul(dev_bf16(x), *d, y)),
                        (K, lambda y: w4.w4a16_mx_matmul_backward(dev_bf16(dy), *d, y))):
        buf = torch.full((M + 40, width), 7.0, dtype=torch.bfloat16, device="cuda")
        call(buf[8:8 + M])
        assert (buf[:8] == 7).all() and (buf[8 + M:] == 7).all()


@pytest.mark.parametrize("M", [1, 5, 20, 40, 130])
def test_not_a_number_stays_in_its_row(M):
    rng = np.random.default_rng(13)
    N, K = 48, 96
    wq, s = ref.random_stored(rng, N, K, 126, 128)
    x = whole(rng, M, K)
    x[0, 33], x[M // 2, 5] = np.inf, np.nan
    s[7, 1] = 255
    w = ref.values(wq, s)
    with np.errstate(invalid="ignore"):
        want = (x[:, None, :] * w[None]).sum(-1)
    same(host(w4.w4a16_mx_matmul(dev_bf16(x), *dev(wq, s))), ref.bf16(want))
    # backward: row 7 of W reaches every dx of its block of K, no other block
    dy = whole(rng, M, N)
    with np.errstate(invalid="ignore"):
        want = (dy[:, :, None] * w[None]).sum(1)
    same(host(w4.w4a16_mx_matmul_backward(dev_bf16(dy), *dev(wq, s))), ref.bf16(want))
    # 4-bit activations: a block that is not a number
    xq, xs = ref.random_stored(rng, M, K, 127, 128)
    xs[M // 2, 2] = 255
    with np.errstate(invalid="ignore"):
        want = (ref.values(xq, xs)[:, None, :] * w[None]).sum(-1)
    same(host(w4.w4a16_mx_matmul_a4(*dev(xq, xs), *dev(wq, s))), ref.bf16(want))


@pytest.mark.parametrize("M", [1, 20, 40, 140])
@pytest.mark.parametrize("e", [0, 1, 60, 128, 129, 200, 252])
def test_scales_over_the_whole_range(M, e):
    """Stored values from 2^-128 to 6 2^125 against x that brings the sums back into range."""
    rng = np.random.default_rng([14, e])
    N, K = 40, 64
    wq, s = ref.random_stored(rng, N, K, e, e)
    a = int(np.clip(120 - e, -100, 100))
    x = whole(rng, M, K) * 2.0 ** a
    w = ref.values(wq, s)
    same(host(w4.w4a16_mx_matmul(dev_bf16(x), *dev(wq, s))), ref.bf16(x @ w.T))
    dy = whole(rng, M, N) * 2.0 ** a
    same(host(w4.w4a16_mx_matmul_backward(dev_bf16(dy), *dev(wq, s))), ref.bf16(dy @ w))
    xq, xs = ref.random_stored(rng, M, K, min(254 - 8, max(1, 247 - e)), min(254 - 8, max(1, 247 - e)))
    same(host(w4.w4a16_mx_matmul_a4(*dev(xq, xs), *dev(wq, s))), ref.bf16(ref.values(xq, xs) @ w.T))


# ------------------------------------------------------------------ streams, graphs, repeats


def test_repeats_bit_for_bit():
    rng = np.random.default_rng(16)
    for M, N, K in ((1, 1000, 2560), (40, 264, 2592), (300, 520, 1056)):
        wq, s = dev(*ref.random_stored(rng, N, K))
        x, dy = dev_bf16(normal(rng, M, K)), dev_bf16(normal(rng, M, N))
        q = w4.w4a16_mx_quantize(x)
        for call in (lambda: w4.w4a16_mx_matmul(x, wq, s), lambda: w4.w4a16_mx_matmul_a4(*q, wq, s),
                     lambda: w4.w4a16_mx_matmul_backward(dy, wq, s)):
            first = call()
            for _ in range(5):
                assert torch.equal(call().view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("M", [1, 24, 150])
def test_block_captured_and_replayed(M):
    """The run of them together, as a fine-tuning step and a prompt use them: forward, backward and the 4-bit
    product captured without a warm-up call, two graphs at once, replayed on new inputs."""
    rng = np.random.default_rng([17, M])
    N, K = 128, 96
    wq, s = ref.random_stored(rng, 2 * N, K, 121, 124)
    dq, ds = ref.random_stored(rng, K, N, 121, 124)        # the projection back to K
    w, wd = ref.values(wq, s), ref.values(dq, ds)
    d, dd = dev(wq, s), dev(dq, ds)
    graphs = []
    for _ in range(2):
        x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        dy = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            h = w4.w4a16_mx_gate_up(x, *d)
            y = w4.w4a16_mx_matmul(h, *dd)
            y4 = w4.w4a16_mx_matmul_a4(*w4.w4a16_mx_quantize(h), *dd)
            dh = w4.w4a16_mx_matmul_backward(dy, *dd)
            dx, dgu = w4.w4a16_mx_gate_up_backward(x, *d, dh)
        graphs.append((g, x, dy, h, y, y4, dh, dx, dgu))
    streams = [torch.cuda.Stream() for _ in graphs]
    for turn in range(3):
        ins = []
        for g, x, dy, *_ in graphs:
            xv, dv = normal(rng, M, K, 0.5), normal(rng, M, K, 0.1)
            x.copy_(dev_bf16(xv))
            dy.copy_(dev_bf16(dv))
            ins.append((xv, dv))
        torch.cuda.synchronize()
        for (g, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (g, x, dy, h, y, y4, dh, dx, dgu), (xv, dv) in zip(graphs, ins):
            near(host(h), *ref.gate_up(xv, w), "h")
            near(host(y), *ref.product(host(h), wd), "y")
            near(host(y4), *ref.product(ref.values(*ref.quantize(host(h))), wd), "y4")
            near(host(dh), *ref.product(dv, wd.T), "dh")
            near(host(dgu), *ref.gate_up_backward(xv, w, host(dh)), "dgu")
            near(host(dx), *ref.product(host(dgu), w.T), "dx")


def test_given_stream():
    """Work on a stream that is given, behind work that is already on it."""
    rng = np.random.default_rng(18)
    M, N, K = 20, 136, 96
    wq, s = ref.random_stored(rng, N, K, 126, 128)
    d = dev(wq, s)
    x = whole(rng, M, K)
    xd = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    src = dev_bf16(x)
    big = torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        for _ in range(20):
            big += 1
        xd.copy_(src)
    y = w4.w4a16_mx_matmul(xd, *d, stream=st)
    q = w4.w4a16_mx_quantize(xd, stream=st)
    y4 = w4.w4a16_mx_matmul_a4(*q, *d, stream=st.cuda_stream)
    st.synchronize()
    w = ref.values(wq, s)
    same(host(y), ref.bf16(x @ w.T))
    same(host(y4), ref.bf16(ref.values(*ref.quantize(x)) @ w.T))


def test_large_offsets():
    """Rows whose byte offsets pass 2^32 in x and 2^31 in y: the last rows against a small call."""
    free = torch.cuda.mem_get_info()[0]
    if free < 24 << 30:
        pytest.skip("needs 24 GB")
    M, N, K = 1_100_000, 2048, 2560
    rng = np.random.default_rng(19)
    wq, s = dev(*ref.random_stored(rng, N, K, 126, 128))
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    tail = dev_bf16(whole(rng, 300, K))
    x[-300:] = tail
    y = w4.w4a16_mx_matmul(x, wq, s)
    assert torch.equal(y[-300:], w4.w4a16_mx_matmul(tail, wq, s))
    assert not y[:1000].any() and not y[M // 2:M // 2 + 1000].any()


def test_refusals_on_the_device():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    wq, s = torch.zeros(16, 8, dtype=torch.int32, device="cuda"), torch.zeros(16, 2, dtype=torch.uint8, device="cuda")
    with pytest.raises(TypeError):
        w4.w4a16_mx_matmul(x.float(), wq, s)
    with pytest.raises(TypeError):
        w4.w4a16_mx_matmul(x, wq.long(), s)
    with pytest.raises(ValueError):
        w4.w4a16_mx_matmul(x, wq, s[:8])
    with pytest.raises(ValueError):
        w4.w4a16_mx_matmul(x[:, ::2], wq, s)
    with pytest.raises(ValueError):
        w4.w4a16_mx_matmul(x, wq, s, torch.empty(4, 8, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(w4.W4A16Error):
        w4.w4a16_mx_quantize(torch.zeros(2, 40, device="cuda"))
    with pytest.raises(ValueError):
        w4.w4a16_mx_gate_up(x, wq[:8], s[:8])
    with pytest.raises(ValueError):
        w4.w4a16_mx_matmul_backward(x, wq, s)
    with pytest.raises(w4.W4A16Error) as e:
        w4.w4a16_mx_matmul_backward(torch.zeros(4, 12, dtype=torch.bfloat16, device="cuda"), wq[:12], s[:12])
    assert e.value.status == w4.ERR_UNSUPPORTED
    with pytest.raises(w4.W4A16Error) as e:
        w4.w4a16_mx_matmul(x.reshape(-1)[8 * 64 // 16:][:64].view(1, 64).flatten()[0:0].new_zeros(65)[1:].view(1, 64), wq, s)
    assert e.value.status == w4.ERR_MISALIGNED


@pytest.mark.parametrize("M", [4, 40])
def test_gate_up_far_out(M):
    """Gates from -200 to 200: no overflow, and only sigmoids below 2^-126 may be lost."""
    K, N = 32, 64                                  # w = 1 at one k of a row: g and u are values of x
    codes = np.zeros((2 * N, K), np.uint32)
    gate = (np.arange(2 * N) // 8) % 2 == 0
    codes[gate, 3] = codes[~gate, 17] = 2
    wq, s = ref.pack(codes), np.full((2 * N, 1), 127, np.uint8)
    x = np.zeros((M, K))
    x[:, 3] = ref.bf16(np.linspace(-200, 200, M) if M > 4 else np.array([-200.0, -88.5, -80.0, 100.0]))
    x[:, 17] = 3.0
    w, dh = ref.values(wq, s), ref.bf16(np.ones((M, N)))
    h, tol = ref.gate_up(x, w)
    lost = 2.0 ** -126 * 3 * (1 + np.abs(x[:, 3:4]))       # |s| < 2^-126 times |u| and the larger factors of it
    near(host(w4.w4a16_mx_gate_up(dev_bf16(x), *dev(wq, s))), h, tol + lost)
    dgu, tol = ref.gate_up_backward(x, w, dh)
    near(host(w4.w4a16_mx_gate_up_backward(dev_bf16(x), *dev(wq, s), dev_bf16(dh))[1]), dgu, tol + lost)


def spread(picked, at, k, stored):
    """Rows of k values that are zeros but for codes picked [rows, len(at)] at columns `at`."""
    rows, words = picked.shape[0], [i // 8 for i in at]
    assert len(set(words)) == len(at)
    if not stored:
        x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
        x[:, at] = dev_bf16(ref.GRID[picked])
        return x
    wq = torch.zeros(rows, k // 8, dtype=torch.int32, device="cuda")
    nibbles = picked.astype(np.uint32) << np.array([4 * (i % 8) for i in at], np.uint32)
    wq[:, words] = torch.from_numpy(nibbles.view(np.int32)).cuda()
    return wq, torch.full((rows, k // 32), 127, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("M,N,K,op", [(2, 2, 2 ** 31 - 65536 - 32, "matmul"), (2, 2, 2 ** 31 - 65536 - 32, "a4"),
                                      (40, 8, 2 ** 26, "matmul"), (40, 16, 2 ** 26, "gate_up"),
                                      (40, 8, 2 ** 26, "backward")])
def test_long_rows(M, N, K, op):
    """Up to the longest rows: offsets beyond 2^32 bytes, and a tile that takes seconds."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    at = [0, 39, K // 2 + 8, K - 40, K - 1]
    rng = np.random.default_rng([21, M, N])
    px, pw = rng.integers(0, 16, (M, len(at))), rng.integers(0, 16, (N, len(at)))
    x, w = ref.GRID[px], ref.GRID[pw]
    wq, s = spread(pw, at, K, True)
    if op == "matmul":
        same(host(w4.w4a16_mx_matmul(spread(px, at, K, False), wq, s)), ref.bf16(x @ w.T))
    elif op == "a4":
        same(host(w4.w4a16_mx_matmul_a4(*spread(px, at, K, True), wq, s)), ref.bf16(x @ w.T))
    elif op == "gate_up":
        h, tol = ref.gate_up(x, w)
        near(host(w4.w4a16_mx_gate_up(spread(px, at, K, False), wq, s)), h, tol)
    else:
        dy = whole(rng, M, N)
        dx = w4.w4a16_mx_matmul_backward(dev_bf16(dy), wq, s)
        same(host(dx[:, at]), ref.bf16(dy @ w))
        dx[:, at] = 0
        assert not dx.any()
    torch.cuda.synchronize()
    assert w4.w4a16_device_status() == 0
