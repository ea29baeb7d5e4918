"""GPU: the layer of examples/decay_block.py, the new operators between the ones that were there: a prompt and then
tokens against the whole prompt, a training run, and its gradients against differences of the loss."""
import importlib.util
import os

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decay_block", os.path.join(ROOT, "examples", "decay_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_prompt_then_tokens_and_training(example):
    diff, losses = example.run()
    # bf16 values all along (about ten roundings of 2^-9 between input and output, of values near the largest)
    assert diff < 2e-2
    assert losses[-1] < 0.97 * losses[0] and all(b < a + 1e-3 for a, b in zip(losses, losses[1:]))


def plain_layer(layer, x, n):
    """The layer's prompt from empty caches in fp64, elementary torch operations: what autograd differentiates."""
    import torch.nn.functional as F
    L = {k: getattr(layer, k).double().requires_grad_(True)
         for k in ("w_qkv", "w_z", "w_u", "w_o", "taps", "head_norm", "post", "pre", "res_scale")}
    B, T, D = x.shape
    p = F.pad(n @ L["w_qkv"], (0, 0, L["taps"].shape[1] - 1, 0))
    c = F.silu(sum(p[:, i:i + T] * L["taps"][:, i] for i in range(L["taps"].shape[1])))
    Hv, d = layer.log_decay.numel(), L["head_norm"].numel()
    Hqk = (c.shape[-1] // d - Hv) // 2
    q, k, v = c.split([Hqk * d, Hqk * d, Hv * d], -1)
    q, k = (t.unflatten(-1, (Hqk, d)).repeat_interleave(Hv // Hqk, 2) for t in (q, k))
    t = torch.arange(T, device=x.device, dtype=torch.float64)
    gap = t[:, None] - t
    decay = torch.where(gap >= 0, torch.exp(layer.log_decay.double()[:, None, None] * gap.clamp(min=0)), 0.0)
    scores = torch.einsum("bthd,bshd->bhts", q, k) * decay * layer.scale
    o = torch.einsum("bhts,bshd->bthd", scores, v.unflatten(-1, (Hv, d)))
    norm = lambda y: y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6)   # noqa: E731
    y = norm(o) * L["head_norm"] * F.silu((n @ L["w_z"]).unflatten(-1, (Hv, d)))
    r = x + L["res_scale"] * torch.sigmoid(n @ L["w_u"]) * norm(y.flatten(-2) @ L["w_o"]) * L["post"]
    return L, r, norm(r) * L["pre"]


def test_layer_gradients_equal_autograd_of_the_plain_layer(example):
    """Relative 2-norm.  About a dozen bf16 roundings (rms 2^-9.2 each, partly averaged out in the sums over 200
    tokens) lie between a weight and the loss: under 1 per cent forward, a few per cent for a gradient that is
    itself a difference of larger terms: 5e-2; a missing or wrong factor would be tens of per cent."""
    layer = example.Layer(3)
    gen = torch.Generator().manual_seed(4)
    x, n = (torch.randn(1, 200, example.D, generator=gen).to("cuda", torch.bfloat16) for _ in range(2))
    gr, gn = (torch.randn(1, 200, example.D, generator=gen).to("cuda", torch.bfloat16) for _ in range(2))
    (r, out), _ = layer.prompt(x, n, layer.empty_cache(1))
    got = layer.backward(gr, gn)
    L, r64, n64 = plain_layer(layer, x.double(), n.double())
    for a, b in ((r, r64), (out, n64)):
        assert float(((a.double() - b).norm() / b.norm()).detach()) < 2e-2
    want = torch.autograd.grad((r64 * gr.double()).sum() + (n64 * gn.double()).sum(), list(L.values()))
    for (name, _), w in zip(L.items(), want):
        e = float((got[name].double() - w).norm() / w.norm())
        assert e < 5e-2, f"{name}: {e:.3e}"
