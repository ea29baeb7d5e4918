"""GPU: prompts of several equal sequences in segments, and the same sequences one by one, against the fp64 statement;
tolerances as derived in test_gpu_scan."""
import pytest

torch = pytest.importorskip("torch")

from oracle import scan as os_   # noqa: E402

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gated_deltanet_recurrence_03_gb300 as gdn  # noqa: E402
from test_gpu_scan import call, close, make, oracle_args, tol32  # noqa: E402


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,D,G,N", [((1500,) * 3, 24, 1, 16), ((700, 700), 48, 2, 8), ((1100,) * 4, 16, 1, 64)])
def test_batches_in_segments(dtype, lens, D, G, N):
    x, _, _, _ = make(dtype, lens, D, G, N, seed=17)
    y, h = call(x)
    want_y, want_h = os_.forward(**oracle_args(x))
    t32, small = tol32(max(lens)), 2.0 ** -8 if dtype == "bf16" else None
    close(want_y, y, small or t32, "y", (0, 1))
    close(want_h, h, t32, "h_final", (2,))
    for i in range(len(lens)):
        one = {k: (v[i:i + 1] if k in ("u", "delta", "B", "C", "z", "h0") else v) for k, v in x.items()}
        yi, hi = call(one)
        close(want_y[i:i + 1], yi, small or t32, "y", (0, 1))
        close(want_h[i:i + 1], hi, t32, "h_final", (2,))
