"""GPU: gradients for rates A = -exp(A_log) that fp32 cannot hold: nothing of a state is left after a token, and as in 64
bits (-exp(A_log) times a sum that is 0) their dA_log is 0."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gated_deltanet_recurrence_03_gb300 as gdn  # noqa: E402
from oracle import scan as osc  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [8, 16])
def test_gradients_of_rates_beyond_fp32(N, dtype):
    gen = torch.Generator().manual_seed(14)
    T, D, f32 = 75, 24, torch.float32
    r = lambda *s, dt=dtype: torch.randn(*s, generator=gen).cuda().to(dt)   # noqa: E731
    u, delta, B, C, z, gy = r(1, T, D), r(1, T, D), r(1, T, 1, N), r(1, T, 1, N), r(1, T, D), r(1, T, D)
    A_log, skip, bias, h0 = 0.5 * r(D, N, dt=f32), r(D, dt=f32), r(D, dt=f32), r(1, D, N, dt=f32)
    beyond = {(3, 0): 88.8, (3, 5): 89.0, (5, 2): 200.0, (7, 7): 700.0}
    for at, v in beyond.items():
        A_log[at] = v
    got = gdn.gdn_selective_scan_bwd(u, delta, A_log, B, C, h0, gy, None, skip=skip, dt_bias=bias, z=z)
    n = lambda t: t.double().cpu().numpy()   # noqa: E731
    want = osc.backward(n(u), n(delta), n(A_log), n(B), n(C), n(gy), n(h0), None, n(skip), n(bias), n(z))
    assert all(torch.isfinite(g).all() for g in got)
    for at in beyond:
        assert want[2][at] == 0 and got[2][at] == 0, at
    # the others as ever: 4 (4 + sqrt(T)) 2^-21 of the largest value (two scans and the sums over tokens)
    assert np.abs(n(got[2]) - want[2]).max() <= 4 * (4 + T ** 0.5) * 2.0 ** -21 * np.abs(want[2]).max()
