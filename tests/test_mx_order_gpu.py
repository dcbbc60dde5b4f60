"""MXFP4 calls back to back on the same buffers: every kernel begins before the one in front of it has
ended, and has to see what that one wrote, not what the buffers held a call earlier.  The results have
to equal, bit for bit, those of the same calls made one at a time on buffers of their own."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import decode_w4a16_g128_b200 as w4  # noqa: E402

TURNS = 24


def inputs(M, N, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(M * 1000003 + N * 1009 + K)
    normal = lambda r, c: torch.randn(r, c, generator=g, device="cuda")
    return [(normal(M, K).bfloat16(), normal(N, K) * 0.1, normal(M, N).bfloat16()) for _ in range(3)]


def apart(sets):
    """Each set's results, every call on new buffers and waited for."""
    out = []
    for x, w, dy in sets:
        q = w4.w4a16_mx_quantize(w)
        torch.cuda.synchronize()
        xq = w4.w4a16_mx_quantize(x)
        torch.cuda.synchronize()
        r = [w4.w4a16_mx_matmul_a4(*xq, *q)]
        torch.cuda.synchronize()
        r.append(w4.w4a16_mx_matmul(x, *q))
        torch.cuda.synchronize()
        r.append(w4.w4a16_mx_gate_up(x, *q))
        torch.cuda.synchronize()
        r.append(w4.w4a16_mx_matmul_backward(dy, *q))
        torch.cuda.synchronize()
        r.append(w4.w4a16_mx_dequantize(*q))
        torch.cuda.synchronize()
        out.append(r)
    return out


def chain(sets, turns, xq, wq, y):
    """Quantise into the same buffers, read them at once, turn after turn."""
    got = []
    for t in range(turns):
        x, w, dy = sets[t % 3]
        r = []
        w4.w4a16_mx_quantize(w, *wq)
        w4.w4a16_mx_quantize(x, *xq)
        r.append(w4.w4a16_mx_matmul_a4(*xq, *wq, y).clone() if t % 2 else w4.w4a16_mx_matmul_a4(*xq, *wq))
        w4.w4a16_mx_quantize(w, *wq)
        r.append(w4.w4a16_mx_matmul(x, *wq))
        w4.w4a16_mx_quantize(w, *wq)
        r.append(w4.w4a16_mx_gate_up(x, *wq))
        w4.w4a16_mx_quantize(w, *wq)
        r.append(w4.w4a16_mx_matmul_backward(dy, *wq))
        w4.w4a16_mx_quantize(w, *wq)
        r.append(w4.w4a16_mx_dequantize(*wq))
        got.append(r)
    return got


# row kernels, tensor-core kernels alone and in pairs, one CTA of work and more than the SMs
SIZES = [(1, 48, 160), (4, 1024, 2560), (8, 9728, 2560), (16, 2560, 2560), (40, 1008, 4064), (100, 4096, 544),
         (300, 2048, 2560), (600, 9728, 608)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_buffers_used_again_at_once(M, N, K):
    sets = inputs(M, N, K)
    want = apart(sets)
    xq, wq = w4.w4a16_mx_quantize(torch.zeros_like(sets[0][0])), w4.w4a16_mx_quantize(torch.zeros_like(sets[0][1]))
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    got = chain(sets, TURNS, xq, wq, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = chain(sets, 6, xq, wq, y)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    for results in (got, again):
        for t, r in enumerate(results):
            for i, (a, b) in enumerate(zip(r, want[t % 3])):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16)), (t, i)
    assert w4.w4a16_device_status() == w4.OK


@pytest.mark.parametrize("M,N,K", SIZES)
def test_products_that_feed_each_other(M, N, K):
    """y of one call is x of the next, in buffers that every turn writes anew."""
    sets = inputs(M, N, K)
    down = w4.w4a16_mx_quantize(torch.randn(K, N // 2, device="cuda") * 0.1) if N // 2 % 32 == 0 else None
    h, xq = torch.empty(M, N // 2, dtype=torch.bfloat16, device="cuda"), w4.w4a16_mx_quantize(sets[0][0])
    want, got = [], []
    stored = [w4.w4a16_mx_quantize(w) for _, w, _ in sets]
    for (x, _, dy), q in zip(sets, stored):
        torch.cuda.synchronize()
        a = w4.w4a16_mx_gate_up(x, *q)
        torch.cuda.synchronize()
        b = w4.w4a16_mx_matmul(a, *down) if down else a
        torch.cuda.synchronize()
        want.append((b, w4.w4a16_mx_matmul_a4(*w4.w4a16_mx_quantize(x), *q)))
    torch.cuda.synchronize()
    for t in range(TURNS):
        x, q = sets[t % 3][0], stored[t % 3]
        w4.w4a16_mx_gate_up(x, *q, h)
        b = w4.w4a16_mx_matmul(h, *down) if down else h.clone()
        w4.w4a16_mx_quantize(x, *xq)
        got.append((b, w4.w4a16_mx_matmul_a4(*xq, *q)))
    torch.cuda.synchronize()
    for t, r in enumerate(got):
        for i, (a, b) in enumerate(zip(r, want[t % 3])):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), (t, i)
