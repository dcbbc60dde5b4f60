"""Layers back to back on the same buffers, on the tensor-core path: each begins before the one in front
of it has ended, and has to see that one's outputs and not what the buffer held a turn earlier.  Equal bit
for bit to the same calls made one at a time on buffers of their own."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import decode_w4a16_g128_b200 as w4  # noqa: E402


def layer(g, n, k):
    return w4.w4a16_quantize(torch.randn(n, k, generator=g, device="cuda") * 0.05)


@pytest.mark.parametrize("M,N,K", [(40, 1024, 2560), (129, 1000, 256), (300, 2560, 1024), (512, 384, 9728)])
def test_layers_that_feed_each_other(M, N, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    N -= N % 128
    ups = [layer(g, N, K) for _ in range(3)]
    downs = [layer(g, K, N) for _ in range(3)]
    xs = [torch.randn(M, K, generator=g, device="cuda").bfloat16() for _ in range(3)]
    want = []
    for x, up, down in zip(xs, ups, downs):
        h = w4.w4a16_matmul(x, *up)
        torch.cuda.synchronize()
        want.append(w4.w4a16_matmul(h, *down))
        torch.cuda.synchronize()
    h, y = (torch.empty(M, n, dtype=torch.bfloat16, device="cuda") for n in (N, K))

    def chain(turns):
        got = []
        for t in range(turns):
            w4.w4a16_matmul(xs[t % 3], *ups[t % 3], h)
            got.append(w4.w4a16_matmul(h, *downs[t % 3], y).clone() if t % 2 else w4.w4a16_matmul(h, *downs[t % 3]))
        return got

    got = chain(24)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        chain(1)                                   # the stream's workspace, before the capture
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        again = chain(6)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    for results in (got, again):
        for t, r in enumerate(results):
            assert torch.equal(r.view(torch.int16), want[t % 3].view(torch.int16)), t
    assert w4.w4a16_device_status() == w4.OK
