"""The gated block's gradients where its sums are empty (K = 0): the formula's values, which are zeros
only where dh is finite."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import decode_w4a16_g128_b200 as w4  # noqa: E402
import mx_reference as ref  # noqa: E402


@pytest.mark.parametrize("M,N", [(1, 8), (3, 16), (150, 1000), (2048, 2056)])
def test_gradients_of_empty_sums(M, N):
    rng = np.random.default_rng([40, M, N])
    dh = ref.bf16(rng.standard_normal((M, N)))
    dh[0, 1], dh[M // 2, N - 1], dh[M - 1, 3] = np.nan, np.inf, -np.inf
    x = torch.empty(M, 0, dtype=torch.bfloat16, device="cuda")
    wq, s = torch.empty(2 * N, 0, dtype=torch.int32, device="cuda"), torch.empty(2 * N, 0, dtype=torch.uint8, device="cuda")
    buf = torch.full((M + 2, 2 * N), 7.0, dtype=torch.bfloat16, device="cuda")
    dx, dgu = w4.w4a16_mx_gate_up_backward(x, wq, s, torch.from_numpy(dh).float().cuda().bfloat16(), dgu=buf[1:M + 1])
    with np.errstate(invalid="ignore"):
        want, _ = ref.gate_up_backward(np.zeros((M, 0)), np.zeros((2 * N, 0)), dh)
    got = dgu.double().cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True) and np.isnan(want).any()
    assert dx.shape == (M, 0) and (buf[0] == 7).all() and (buf[-1] == 7).all()
