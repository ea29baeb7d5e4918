"""GPU: gradients of many short packed sequences of a wide layer: each sequence's are those of a call of its own, and the
scratch stays near the tensors' size."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gated_deltanet_recurrence_03_gb300 as gdn  # noqa: E402


@pytest.mark.parametrize("lens", [[9] * 512, [1, 0, 33, 8, 7, 64, 2] * 60, [3] * 100 + [2000] + [5] * 100], ids=["9s", "mixed", "one long"])
def test_gradients_of_many_short_sequences(lens):
    D, N, n, T = 4096, 16, len(lens), sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(15)
    r = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=gen, device="cuda", dtype=dt)   # noqa: E731
    u, delta, z, gy, B, C = r(1, T, D), r(1, T, D), r(1, T, D), r(1, T, D), r(1, T, 1, N), r(1, T, 1, N)
    f32 = torch.float32
    A_log, skip, bias = r(D, N, dt=f32), r(D, dt=f32), r(D, dt=f32) - 3
    h0, gh = r(n, D, N, dt=f32), r(n, D, N, dt=f32)
    starts = [sum(lens[:i]) for i in range(n + 1)]
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    parts = dict(skip=skip, dt_bias=bias)
    gdn.gdn_selective_scan_bwd(u[:, :8].contiguous(), delta[:, :8].contiguous(), A_log, B[:, :8].contiguous(),
                               C[:, :8].contiguous(), None, gy[:, :8].contiguous(), z=z[:, :8].contiguous(), **parts)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    got = gdn.gdn_selective_scan_bwd(u, delta, A_log, B, C, h0, gy, gh, z=z, cu_seqlens=cu, **parts)
    torch.cuda.synchronize()
    state = D * N * 4
    # a state for every 8 tokens, four for every sequence, three for every 32 tokens, 4 D N / 128 sums of B and C for every token;
    # the gradients themselves (a state for every sequence, six tensors of tokens)
    assert torch.cuda.max_memory_allocated() - before <= 1.1 * (state * (T / 8 + 4 * n + 3 * T / 32 + n) + state * T / 32 + 7 * T * D * 2) + (64 << 20)
    for i in [*range(0, n, max(1, n // 12)), 100, n - 1]:
        s = slice(starts[i], starts[i + 1])
        if s.start == s.stop:
            assert torch.equal(got[8][i], gh[i])
            continue
        cut = lambda t: t[:, s].contiguous()   # noqa: E731
        one = gdn.gdn_selective_scan_bwd(cut(u), cut(delta), A_log, cut(B), cut(C), h0[i:i + 1], cut(gy), gh[i:i + 1], z=cut(z), **parts)
        for name, k in (("u", 0), ("delta", 1), ("B", 3), ("C", 4), ("z", 7)):
            a, b = got[k][:, s].double(), one[k].double()
            # other segments, other sums of decays: the fp32 results differ by roundings, the bf16 ones by a step at most
            assert float((a - b).abs().max()) <= 2.0 ** -7 * float(b.abs().max()), (name, i)
        assert float((got[8][i] - one[8][0]).abs().max()) <= 2.0 ** -21 * 4 * (4 + lens[i] ** 0.5) * float(one[8].abs().max())
