"""The convolution's binding enters the context of a given stream before it allocates: a stream of another device is refused
there (no GPU needed), as in every operator whose results belong to the stream that its kernels run on."""
import pytest

torch = pytest.importorskip("torch")
pytest.importorskip("gated_deltanet_recurrence_03_gb300._lib")
from gated_deltanet_recurrence_03_gb300 import api   # noqa: E402


class Elsewhere:
    device = torch.device("cuda", 7)
    cuda_stream = 0


@pytest.fixture(scope="module", autouse=True)
def lib():
    from gated_deltanet_recurrence_03_gb300 import build
    build.build()


x, w, bias, cache = torch.zeros(1, 8, 64), torch.zeros(64, 4), torch.zeros(64), torch.zeros(1, 3, 64)
CALLS = {
    "fwd": lambda s: api.gdn_causal_conv1d_fwd(x, w, cache, bias=bias, stream=s),
    "bwd": lambda s: api.gdn_causal_conv1d_bwd(x, w, x, cache, bias=bias, stream=s),
    "step": lambda s: api.gdn_causal_conv1d_step(x[:, 0], w, cache, bias=bias, stream=s),
    "fwd qkv": lambda s: api.gdn_causal_conv1d_fwd_qkv(x, w, (16, 16, 32), cache, bias=bias, stream=s),
    "step qkv": lambda s: api.gdn_causal_conv1d_step_qkv(x[:, 0], w, cache, (16, 16, 32), bias=bias, stream=s),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_stream_comes_before_what_the_call_allocates(name, monkeypatch):
    made = []
    for f in ("empty", "zeros"):
        monkeypatch.setattr(torch, f, lambda *a, f=getattr(torch, f), **k: made.append(a) or f(*a, **k))
    with pytest.raises(ValueError, match="stream is on"):
        CALLS[name](Elsewhere())
    assert not made
