"""The microscaled 4-bit operators of this package, as they are measured.

The format (MXFP4): blocks of 32 values along K share a power-of-two scale 2^(e - 127), stored as
one byte e (255: the block is not a number); each value is a 4-bit code, sign, two exponent bits
and one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives.  Eight codes a word, the
lowest k in the lowest bits: codes int32 [rows, K/8], scales uint8 [rows, K/32].

Operators: `quantize` (weights or activations to the format, and back to values), `matmul` (BF16
activations times stored weights), `matmul_a4` (activations quantised on the way, both operands in
4 bits), `gate_up` (a gated feed-forward block's two projections, the activation and the product:
h = silu(x Wg^T) * (x Wu^T)), `matmul_backward` (dx = dy W) and `gate_up_backward` (from x and dh,
the gradients of both projections' outputs and of x).  The gate and up rows are interleaved in
blocks of eight, as in the package's w4a16_gate_up.
"""
import math

import torch

own = False

BLOCK = 32
OPS = ("quantize", "matmul", "matmul_a4", "gate_up", "matmul_backward", "gate_up_backward")

# Sizes: the hidden size 2560 and the feed-forward size 9728 of this repository's benchmark, its
# prefill of 2048 rows and its partial tiles of 509 and 129 rows.
MOST = 2048 * 9728 * 2560


def listed():
    return [
        # one token's activations on their way into a 4-bit product
        {"name": "quantize one token", "op": "quantize", "M": 0, "N": 1, "K": 2560, "dtype": "bf16"},
        # a feed-forward projection's weights, once, when a checkpoint is loaded
        {"name": "quantize weights", "op": "quantize", "M": 0, "N": 9728, "K": 2560, "dtype": "f32"},
        # one decoded token through one projection: latency
        {"name": "matmul decode", "op": "matmul", "M": 1, "N": 9728, "K": 2560, "dtype": "bf16"},
        # a prompt through the same projection
        {"name": "matmul prefill", "op": "matmul", "M": 2048, "N": 9728, "K": 2560, "dtype": "bf16"},
        # a short prompt, ragged in every size: an odd number of outputs, a last block of K alone
        {"name": "a4 ragged", "op": "matmul_a4", "M": 77, "N": 1001, "K": 4064, "dtype": "bf16"},
        # a prompt with both operands in 4 bits
        {"name": "a4 prefill", "op": "matmul_a4", "M": 2048, "N": 9728, "K": 2560, "dtype": "bf16"},
        # five sequences decoded together through the gated block
        {"name": "gate_up decode", "op": "gate_up", "M": 5, "N": 9728, "K": 2560, "dtype": "bf16"},
        # an odd chunk of a prompt through the gated block
        {"name": "gate_up chunk", "op": "gate_up", "M": 509, "N": 9728, "K": 2560, "dtype": "bf16"},
        # the input's gradient of a small layer, partial tiles everywhere
        {"name": "backward ragged", "op": "matmul_backward", "M": 129, "N": 1000, "K": 2592, "dtype": "bf16"},
        # the input's gradient of a feed-forward projection, a training batch of 2048 tokens
        {"name": "backward batch", "op": "matmul_backward", "M": 2048, "N": 9728, "K": 2560, "dtype": "bf16"},
        # fine-tuning with few tokens: latency of the gated block's backward pass
        {"name": "gate_up backward few", "op": "gate_up_backward", "M": 64, "N": 9728, "K": 2560, "dtype": "bf16"},
        # the gated block's backward pass, a training batch of 1024 tokens
        {"name": "gate_up backward", "op": "gate_up_backward", "M": 1024, "N": 9728, "K": 2560, "dtype": "bf16"},
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(OPS)
    while True:
        m = _between(rng, 1, 2048)
        n = _between(rng, 8, 9728)
        k = 32 * _between(rng, 1, 304)
        if op == "quantize":
            n = _between(rng, 1, 9728)
            m = 0
        if op in ("gate_up", "gate_up_backward", "matmul_backward"):
            n = max(8, n // 8 * 8)
        cost = max(m, 1) * n * k * {"gate_up": 2, "gate_up_backward": 4}.get(op, 1)
        if n * k <= 9728 * 2560 and cost <= 2 * MOST:
            return {"op": op, "M": m, "N": n, "K": k, "dtype": rng.choice(("bf16", "f32")) if op == "quantize" else "bf16"}


# ------------------------------------------------------------------ the format, in plain operations


def _encode(w):
    """Values [rows, K] -> (codes int32 [rows, K/8], scales uint8 [rows, K/32])."""
    rows, k = w.shape
    b = w.float().reshape(rows, k // BLOCK, BLOCK)
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    e = ((top.view(torch.int32) >> 23) - 2).clamp(min=0)            # floor(log2 top) - 2 + 127
    s = b.abs().double() * torch.exp2(127.0 - e.double())[..., None]
    # nearest value of the grid, ties to the even code, above 6 down to 6
    c = ((s > 0.25).int() + (s >= 0.75).int() + (s > 1.25).int() + (s >= 1.75).int() + (s > 2.5).int()
         + (s >= 3.5).int() + (s > 5.0).int())
    c = c + 8 * torch.signbit(b).int()
    c = torch.where(bad[..., None], 0, c)
    e = torch.where(bad, 255, e)
    words = (c.reshape(rows, k // 8, 8).long() << (4 * torch.arange(8, device=w.device))).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words)
    return words.int(), e.to(torch.uint8)


def _decode(words, scales):
    """The values in 32 bits (every one of them is exact in BF16 too)."""
    rows, n = words.shape
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=words.device)
    grid = torch.cat([grid, -grid])
    c = (words[..., None] >> (4 * torch.arange(8, device=words.device, dtype=torch.int32))) & 15
    v = grid[c.reshape(rows, n * 8 // BLOCK, BLOCK)]
    e = scales.double()
    f = torch.where(scales == 255, torch.full_like(e, math.nan), torch.exp2(e - 127.0))
    return (v.double() * f[..., None]).float().reshape(rows, n * 8)


def _halves(w):
    """Rows interleaved in blocks of eight -> gate rows, up rows."""
    b = w.reshape(w.shape[0] // 16, 2, 8, *w.shape[1:])
    return b[:, 0].reshape(w.shape[0] // 2, *w.shape[1:]), b[:, 1].reshape(w.shape[0] // 2, *w.shape[1:])


# ------------------------------------------------------------------ states


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    m, n, k, op = case["M"], case["N"], case["K"], case["op"]
    s = {"op": op}

    def normal(rows, cols, scale):
        return torch.randn(rows, cols, generator=g, device="cuda") * scale

    def activations(rows, cols):
        # one value in a hundred is an outlier, twenty times as large
        x = normal(rows, cols, 1.0)
        out = torch.rand(rows, cols, generator=g, device="cuda") < 0.01
        return torch.where(out, 20.0 * x, x).bfloat16()

    if op == "quantize":
        s["w"] = normal(n, k, 0.02) if case["dtype"] == "f32" else activations(n, k)
        return s
    rows = 2 * n if op in ("gate_up", "gate_up_backward") else n
    s["wq"], s["scales"] = _encode(normal(rows, k, 0.02))
    if op == "matmul_backward":
        s["dy"] = normal(m, n, 0.01).bfloat16()
        return s
    s["x"] = activations(m, k)
    if op == "gate_up_backward":
        s["dh"] = normal(m, n, 0.01).bfloat16()
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import decode_w4a16_g128_b200 as w4

    op = s["op"]
    if op == "quantize":
        return w4.w4a16_mx_dequantize(*w4.w4a16_mx_quantize(s["w"]))
    if op == "matmul":
        return w4.w4a16_mx_matmul(s["x"], s["wq"], s["scales"])
    if op == "matmul_a4":
        return w4.w4a16_mx_matmul_a4(*w4.w4a16_mx_quantize(s["x"]), s["wq"], s["scales"])
    if op == "gate_up":
        return w4.w4a16_mx_gate_up(s["x"], s["wq"], s["scales"])
    if op == "matmul_backward":
        return w4.w4a16_mx_matmul_backward(s["dy"], s["wq"], s["scales"])
    dx, dgu = w4.w4a16_mx_gate_up_backward(s["x"], s["wq"], s["scales"], s["dh"])
    return {"dx": dx, "dgu": dgu}


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _decode(*_encode(s["w"])).bfloat16()
    w = _decode(s["wq"], s["scales"])
    if op == "matmul":
        return (s["x"].float() @ w.T).bfloat16()
    if op == "matmul_a4":
        return (_decode(*_encode(s["x"])) @ w.T).bfloat16()
    if op == "matmul_backward":
        return (s["dy"].float() @ w).bfloat16()
    wg, wu = _halves(w)
    x = s["x"].float()
    g, u = x @ wg.T, x @ wu.T
    t = 1.0 / (1.0 + torch.exp(-g))
    if op == "gate_up":
        return (g * t * u).bfloat16()
    dh = s["dh"].float()
    dg, du = dh * u * t * (1.0 + g * (1.0 - t)), dh * g * t
    m, n = dh.shape
    dgu = torch.stack([dg.reshape(m, n // 8, 8), du.reshape(m, n // 8, 8)], 2).reshape(m, 2 * n)
    return {"dx": (dg @ wg + du @ wu).bfloat16(), "dgu": dgu.bfloat16()}


# ------------------------------------------------------------------ cost and definition


def work(case):
    m, n, k, op = case["M"], case["N"], case["K"], case["op"]
    stored = k / 2 + k / 32                                    # bytes of a row of codes and scales
    if op == "quantize":
        return {"bytes": n * (k * (4 if case["dtype"] == "f32" else 2) + stored + 2 * k), "flops": 2 * n * k}
    if op in ("matmul", "matmul_a4", "matmul_backward"):
        return {"bytes": n * stored + 2 * m * (n + k), "flops": 2 * m * n * k}
    if op == "gate_up":
        return {"bytes": 2 * n * stored + 2 * m * (n + k), "flops": 4 * m * n * k}
    return {"bytes": 2 * n * stored + 2 * m * (n + k) + 2 * m * (2 * n + k), "flops": 8 * m * n * k}


def _exact_round(w):
    """The values that the format stands for, from its definition, in 64 bits."""
    rows, k = w.shape
    b = w.double().reshape(rows, k // 32, 32)
    top = b.abs().amax(-1, keepdim=True)
    _, p = torch.frexp(top)                                     # top = f 2^p with f in [0.5, 1)
    e = torch.where(top > 0, p - 3, torch.full_like(p, -127)).clamp(min=-127)
    unit = torch.ldexp(torch.ones_like(top), e)
    a = (b / unit).abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    v = torch.copysign((torch.round(a / step) * step).clamp(max=6.0), b) * unit
    return torch.where(torch.isfinite(b).all(-1, keepdim=True), v, torch.full_like(v, math.nan)).reshape(rows, k)


def _exact_values(words, scales):
    rows, n = words.shape
    c = torch.stack([(words.long() >> (4 * j)) & 15 for j in range(8)], -1).reshape(rows, -1)
    mant, ex, sign = (c & 1).double(), ((c >> 1) & 3), 1.0 - 2.0 * (c >> 3).double()
    v = torch.where(ex == 0, 0.5 * mant, (1.0 + 0.5 * mant) * torch.exp2(ex.double() - 1.0))
    e = scales.double().repeat_interleave(32, dim=1)
    return torch.where(e == 255, torch.full_like(v, math.nan), sign * v * torch.exp2(e - 127.0))


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantize":
        return _exact_round(s["w"])
    w = _exact_values(s["wq"], s["scales"])
    if op == "matmul":
        return s["x"].double() @ w.T
    if op == "matmul_a4":
        return _exact_round(s["x"]) @ w.T
    if op == "matmul_backward":
        return s["dy"].double() @ w
    x = s["x"].double()
    gu = (x @ w.T).reshape(x.shape[0], -1, 2, 8)
    g, u = gu[:, :, 0], gu[:, :, 1]
    t = torch.sigmoid(g)
    if op == "gate_up":
        return (g * t * u).reshape(x.shape[0], -1)
    dh = s["dh"].double().reshape(g.shape)
    dgu = torch.stack([dh * u * (t + g * t * (1 - t)), dh * g * t], 2).reshape(x.shape[0], -1)
    return {"dx": dgu @ w, "dgu": dgu}
