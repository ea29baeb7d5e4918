"""GPU: what a call with a stream of its own allocates (results, scratch) belongs to that stream: what is still queued on the
current stream in the memory that the allocator hands out does not reach it.  All forms of the convolution."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gated_deltanet_recurrence_03_gb300 as gdn  # noqa: E402


def calls():
    gen = torch.Generator().manual_seed(16)
    n = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()   # noqa: E731
    f = lambda *s: torch.randn(*s, generator=gen).cuda()   # noqa: E731
    x, dy, w, bias, cache = n(1, 640, 512), n(1, 640, 512), f(512, 4), f(512), n(1, 3, 512)

    def each(t):
        """Updated in place: a copy for every call, made before any stream is given."""
        return [t.clone() for _ in range(4)]
    caches, qkv_caches = each(n(640, 3, 512)), each(n(640, 3, 512))
    return {
        "conv": lambda **s: gdn.gdn_causal_conv1d_fwd(x, w, cache, bias=bias, **s),
        "conv bwd": lambda **s: gdn.gdn_causal_conv1d_bwd(x, w, dy, cache, bias=bias, **s),
        "conv bwd without a bias": lambda **s: gdn.gdn_causal_conv1d_bwd(x, w, dy, cache, **s),
        "conv step": lambda **s: (gdn.gdn_causal_conv1d_step(x[0], w, caches.pop(), bias=bias, **s),),
        "conv qkv": lambda **s: gdn.gdn_causal_conv1d_fwd_qkv(x, w, (128, 128, 256), cache, bias=bias, **s),
        "conv step qkv": lambda **s: gdn.gdn_causal_conv1d_step_qkv(x[0], w, qkv_caches.pop(), (128, 128, 256), bias=bias, **s),
    }


def flat(r):
    return [t for x in r for t in (flat(x) if isinstance(x, (tuple, list)) else [x]) if t is not None]


@pytest.mark.parametrize("name", ["conv", "conv bwd", "conv bwd without a bias", "conv step", "conv qkv", "conv step qkv"])
def test_new_tensors_are_not_in_use_on_another_stream(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = [t.clone() for t in flat(call())]
    torch.cuda.synchronize()
    flat(call(stream=side))   # its memory is in the allocator's pools from here on
    torch.cuda.synchronize()
    blocks = [torch.empty_like(t) for t in want for _ in range(4)]
    torch.cuda._sleep(100_000_000)   # tens of milliseconds before the writes below
    for t in blocks:
        t.fill_(7.0)
    del blocks, t
    got = flat(call(stream=side))
    torch.cuda.synchronize()
    for w, r in zip(want, got):
        assert torch.equal(w, r), name
