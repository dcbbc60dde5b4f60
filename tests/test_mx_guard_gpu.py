"""Nothing outside the outputs is written: every MXFP4 operator into the middle of a buffer of known
bytes, at sizes that end inside tiles, words' vectors and stores (odd numbers of outputs among them), on
both sides of each limit between kernels.  What is written has to be right as well: whole numbers, equal
bit for bit, where the operator's sums can be, else the plain call's result."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import decode_w4a16_g128_b200 as w4  # noqa: E402
import mx_reference as ref  # noqa: E402

BAND = 4096                       # guard bytes on each side, a multiple of 16


class Guarded:
    """A tensor in the middle of a buffer whose other bytes are 0xA5; `odd`: its start is a multiple of 16
    bytes and not of 32."""

    def __init__(self, rows, cols, dtype, odd):
        size = rows * cols * torch.empty((), dtype=dtype).element_size()
        lo = BAND + (16 if odd else 0)
        self.buf = torch.full((lo + size + BAND,), 0xA5, dtype=torch.uint8, device="cuda")
        assert self.buf.data_ptr() % 32 == 0
        self.lo, self.hi = lo, lo + size
        self.t = self.buf[lo:lo + size].view(dtype).view(rows, cols)

    def check(self):
        assert (self.buf[:self.lo] == 0xA5).all(), "written in front of the output"
        assert (self.buf[self.hi:] == 0xA5).all(), "written behind the output"


def whole(rng, rows, k):
    x = torch.from_numpy(rng.integers(-8, 9, (rows, k)).astype(np.float32)).cuda()
    return x.bfloat16(), x.double()


def stored(rng, rows, k, lo=126, hi=128):
    wq, s = ref.random_stored(rng, rows, k, lo, hi)
    wq, s = torch.from_numpy(wq.view(np.int32).copy()).cuda(), torch.from_numpy(s.copy()).cuda()
    return wq, s, w4.w4a16_mx_dequantize(wq, s, dtype=torch.float32).double()


def same(got, want):
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


ROWS = [1, 5, 8, 9, 16, 17, 31, 33, 77, 127, 128, 129, 257]


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("N", [1, 8, 33, 136, 1001])
@pytest.mark.parametrize("M", ROWS)
def test_products(M, N, odd):
    rng = np.random.default_rng([60, M, N])
    K = 160
    wq, s, w = stored(rng, N, K)
    x, xd = whole(rng, M, K)
    y = Guarded(M, N, torch.bfloat16, odd)
    w4.w4a16_mx_matmul(x, wq, s, y.t)
    same(y.t, (xd @ w.T).float().bfloat16())
    y.check()
    xq, xs, v = stored(rng, M, K, 127, 128)
    y = Guarded(M, N, torch.bfloat16, odd)
    w4.w4a16_mx_matmul_a4(xq, xs, wq, s, y.t)
    same(y.t, (v @ w.T).float().bfloat16())
    y.check()
    if N % 8 == 0:
        dy, dyd = whole(rng, M, N)
        dx = Guarded(M, K, torch.bfloat16, odd)
        w4.w4a16_mx_matmul_backward(dy, wq, s, dx.t)
        same(dx.t, (dyd @ w).float().bfloat16())
        dx.check()


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("N", [8, 24, 136, 1000])
@pytest.mark.parametrize("M", ROWS)
def test_gated_block(M, N, odd):
    rng = np.random.default_rng([61, M, N])
    K = 96
    wq, s, w = stored(rng, 2 * N, K, 119, 121)
    x, xd = whole(rng, M, K)
    dh, _ = whole(rng, M, N)
    h, dx, dgu = (Guarded(M, n, torch.bfloat16, odd) for n in (N, K, 2 * N))
    w4.w4a16_mx_gate_up(x, wq, s, h.t)
    w4.w4a16_mx_gate_up_backward(x, wq, s, dh, dx.t, dgu.t)
    same(h.t, w4.w4a16_mx_gate_up(x, wq, s))
    for got, want in zip((dx.t, dgu.t), w4.w4a16_mx_gate_up_backward(x, wq, s, dh)):
        same(got, want)
    g, u = ((xd @ w.T).reshape(M, -1, 2, 8)[:, :, i].reshape(M, N) for i in (0, 1))      # exact in FP32
    want = g * torch.sigmoid(g) * u
    err = ((4 + 1.173 * g.abs()) * 2.0 ** -23 + 12 * 2.0 ** -24) * want.abs()            # see mx_reference.scalar
    assert ((h.t.double() - want).abs() <= ref.HALF_STEP * (want.abs() + err) + err + ref.TINY).all()
    for t in (h, dx, dgu):
        t.check()


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,K", [(1, 32), (1, 96), (3, 32), (5, 1056), (7, 4064), (129, 160), (1, 32800), (257, 2592),
                                 (1031, 8224)])
def test_conversions(N, K, dtype, odd):
    """Sizes on both sides of a CTA's and a grid's share, ends inside a thread's group of words."""
    rng = np.random.default_rng([62, N, K])
    wq, s = ref.random_stored(rng, N, K, 110, 140)
    wq, s = torch.from_numpy(wq.view(np.int32).copy()).cuda(), torch.from_numpy(s.copy()).cuda()
    v = Guarded(N, K, dtype, odd)
    w4.w4a16_mx_dequantize(wq, s, v.t)
    grid = torch.from_numpy(ref.GRID).cuda()
    c = (wq.long()[..., None] >> (4 * torch.arange(8, device="cuda"))) & 15
    want = grid[c].reshape(N, K // 32, 32) * torch.exp2(s.double() - 127)[..., None]
    same(v.t, want.reshape(N, K).to(dtype))
    v.check()
    q, e = Guarded(N, K // 8, torch.int32, odd), Guarded(N, K // 32, torch.uint8, odd)
    w4.w4a16_mx_quantize(v.t, q.t, e.t)
    again = w4.w4a16_mx_dequantize(q.t, e.t, dtype=torch.float32).double()
    # values of the format come back unless a block's largest is below 4 units: then all are finer, and exact
    assert torch.equal(again, v.t.double())
    q.check()
    e.check()
