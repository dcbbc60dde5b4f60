"""MXFP4 in plain numpy, 64 bits: the format, the products and the gated block, for the tests.

Tolerances (all derived, none measured).  Every stored value is exact in BF16 and every product
of BF16 values exact in FP32, so an output errs by its FP32 sum and one rounding to BF16:

* the rounding: at most half a step, 2^-8 of the value;
* the sum: the tensor cores add 16 products at a time to a running sum, aligned to the largest and
  cut off below 24 bits (at most 2^-23 of the magnitudes' sum a step, 16 + 1 terms inside one), and the
  warps', splits' or lanes' partial sums join in at most 32 more additions: K/16 + 32 steps of at
  most 2^-23 of S = sum |x w|.  4-bit operands take 64 products a step; the bound covers them.
"""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
GRID = np.concatenate([GRID, -GRID])


def bf16(a):
    """float64/32 -> nearest bfloat16 values (as float64), ties to even, from the exact value."""
    a = np.asarray(a, np.float64)
    m, e = np.frexp(a)                         # |m| in [0.5, 1): 8 significant bits
    q = np.maximum(e - 8, -133)                # last place; -133 is BF16's smallest step
    with np.errstate(invalid="ignore", over="ignore"):
        r = np.ldexp(np.rint(np.ldexp(a, -q)), q)
        r = np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, a), r)
    return np.where(np.isfinite(a), r, a)


def bf16_bits(values):
    """Values that are exact in BF16 -> their bit patterns."""
    return (np.asarray(values, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def pack(codes):
    """Codes 0..15 [rows, K] -> uint32 [rows, K/8], the lowest k in the lowest bits."""
    c = np.asarray(codes, np.uint32).reshape(codes.shape[0], -1, 8)
    return (c << (4 * np.arange(8, dtype=np.uint32))).sum(-1, dtype=np.uint64).astype(np.uint32)


def quantize(w):
    """(codes uint32 [rows, K/8], scales uint8 [rows, K/32]) of w, block by block and value by
    value: the nearest of the eight magnitudes, the even code where two are as near."""
    w = np.asarray(w, np.float64)
    rows, k = w.shape
    codes, scales = np.zeros((rows, k), np.uint32), np.zeros((rows, k // 32), np.uint8)
    for r in range(rows):
        for b in range(k // 32):
            v = w[r, 32 * b:32 * b + 32]
            if not np.isfinite(v).all():
                scales[r, b] = 255
                continue
            top = np.abs(v).max()
            e = max(0, int(np.floor(np.log2(top))) + 125) if top > 0 else 0
            if top > 0 and 2.0 ** (np.floor(np.log2(top)) + 1) <= top:   # log2 rounded down past a power
                e += 1
            scales[r, b] = e
            a = np.abs(v) * 2.0 ** (127 - e)
            d = np.abs(a[:, None] - GRID[None, :8])
            best = d.min(-1, keepdims=True)
            # of the nearest codes (one or two), an even one if there is one
            near = d == best
            pick = np.where(near[:, ::2].any(-1), 2 * near[:, ::2].argmax(-1), near.argmax(-1))
            codes[r, 32 * b:32 * b + 32] = pick + 8 * np.signbit(v)
    return pack(codes), scales


def values(wq, scales):
    """The stored values [rows, K] in 64 bits."""
    rows = wq.shape[0]
    c = (wq[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15
    v = GRID[c].reshape(rows, -1)
    with np.errstate(invalid="ignore"):
        f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
        return v * np.repeat(f, 32, axis=1)


def random_stored(rng, rows, k, lo=118, hi=124):
    """Random codes and scale bytes in [lo, hi]."""
    return (rng.integers(0, 2 ** 32, (rows, k // 8), dtype=np.uint32),
            rng.integers(lo, hi + 1, (rows, k // 32)).astype(np.uint8))


def sum_error(x, w):
    """Bound on the error of the FP32 sums of x . w^T (the module's second bullet)."""
    return (x.shape[1] / 16 + 32) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)


HALF_STEP = 2.0 ** -8
TINY = 2.0 ** -133       # BF16's smallest step: what the rounding of a subnormal may be off by


def product(x, w):
    """(x . w^T, tolerance of a BF16 output)."""
    y, s = x @ w.T, sum_error(x, w)
    return y, HALF_STEP * (np.abs(y) + s) + s + TINY


def interleave(gate, up):
    return np.stack([gate.reshape(gate.shape[0] // 8, 8, -1), up.reshape(up.shape[0] // 8, 8, -1)], 1).reshape(
        2 * gate.shape[0], -1)


def split(a, axis):
    """gate and up parts of an axis interleaved in blocks of 8."""
    a = np.moveaxis(a, axis, -1)
    b = a.reshape(*a.shape[:-1], -1, 2, 8)
    g, u = b[..., 0, :], b[..., 1, :]
    g, u = (np.moveaxis(t.reshape(*a.shape[:-1], -1), -1, axis) for t in (g, u))
    return g, u


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


# FP32 evaluation of the scalar formulas: the exponential's documented bound is 2 + 1.173 |g| steps of
# 2^-23, the division's 2, and at most a dozen more operations are off by 2^-24 of their result each;
# none but 1 + g (1 - s) subtracts, and that one is bounded by its terms.
def scalar(g):
    return (2 + 1.173 * np.abs(g) + 2) * 2.0 ** -23 + 12 * 2.0 ** -24


def gate_up(x, w):
    """(h, tolerance): silu' <= 1.1 carries the sums' error through the product."""
    gu, s = x @ w.T, sum_error(x, w)
    (g, u), (eg, eu) = split(gu, 1), split(s, 1)
    h = g * sigmoid(g) * u
    e = 1.1 * (np.abs(u) + eu) * eg + np.abs(g * sigmoid(g)) * eu + scalar(g) * np.abs(h)
    return h, HALF_STEP * (np.abs(h) + e) + e + TINY


def gate_up_backward(x, w, dh):
    """(dgu, tolerance): |silu'| <= 1.1 and |silu''| <= 0.5."""
    gu, err = x @ w.T, sum_error(x, w)
    (g, u), (eg, eu) = split(gu, 1), split(err, 1)
    s = sigmoid(g)
    dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
    a = np.abs(dh)
    # s (1 + g (1 - s)): its terms' magnitudes bound the cancellation; 1 - s loses 2^-24 absolutely
    edg = a * (0.5 * (np.abs(u) + eu) * eg + 1.1 * eu) + scalar(g) * a * np.abs(u) * s * (1 + 2 * np.abs(g))
    edu = a * 1.1 * eg + scalar(g) * np.abs(du)
    d = np.stack([dg.reshape(len(x), -1, 8), du.reshape(len(x), -1, 8)], 2).reshape(len(x), -1)
    e = np.stack([edg.reshape(len(x), -1, 8), edu.reshape(len(x), -1, 8)], 2).reshape(len(x), -1)
    return d, HALF_STEP * (np.abs(d) + e) + e + TINY
