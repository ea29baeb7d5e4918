"""GPU: results of calls on a stream of their own survive what is still queued on the current stream in the memory
that the allocator hands to them."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def calls():
    import gated_deltanet_recurrence_03_gb300 as gdn
    gen = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()   # noqa: E731
    q, k, v, do = n(1, 640, 2, 64), n(1, 640, 2, 64), n(1, 640, 4, 64), n(1, 640, 4, 64)
    g = -torch.exp2(-torch.linspace(1.0, 9.0, 4)).cuda()
    S = torch.randn(1, 4, 64, 64, generator=gen).cuda()
    states = [S.clone() for _ in range(3)]   # updated in place, one a call
    x, b, u = n(300, 512), n(300, 512), n(300, 512)
    w = torch.ones(512).cuda()
    return {
        "fwd": lambda **o: gdn.gdn_decay_attn_fwd(q, k, v, g, S, **o),
        "bwd": lambda **o: gdn.gdn_decay_attn_bwd(q, k, v, g, S, do, S, **o),
        "step": lambda **o: (gdn.gdn_decay_attn_step(q[:, 0], k[:, 0], v[:, 0], g, states.pop(), **o),),
        "norm": lambda **o: gdn.gdn_block_norm_fwd(x, b, w, w, gate=u, res_scale=w, **o),
        "norm bwd": lambda **o: gdn.gdn_block_norm_bwd(x, b, w, w, x, b, gate=u, res_scale=w, **o),
    }


@pytest.mark.parametrize("name", ["fwd", "bwd", "step", "norm", "norm bwd"])
def test_new_tensors_are_not_in_use_on_another_stream(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in call()]
    call(stream=side)   # its memory is in the allocator's pools from here on
    torch.cuda.synchronize()
    blocks = [torch.empty_like(t) for t in want for _ in range(4)]
    torch.cuda._sleep(100_000_000)   # tens of milliseconds before the writes below
    for t in blocks:
        t.fill_(7.0)
    del blocks, t
    got = call(stream=side)
    torch.cuda.synchronize()
    for w, r in zip(want, got):
        assert torch.equal(w, r), name


def test_stream_of_another_device_is_refused():
    import gated_deltanet_recurrence_03_gb300 as gdn

    class Elsewhere:
        device = torch.device("cuda", 7)
        cuda_stream = 0
    x, w = torch.zeros(2, 64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="stream is on"):
        gdn.gdn_block_norm_fwd(x, x, w, w, stream=Elsewhere())
