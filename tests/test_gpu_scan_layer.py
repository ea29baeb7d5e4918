"""GPU: the layer of examples/scan_block.py, the selective scan and the layer norm around the conv: a prompt and then
tokens against the whole prompt, a training run, and its gradients against autograd of the plain layer."""
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
    spec = importlib.util.spec_from_file_location("scan_block", os.path.join(ROOT, "examples", "scan_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_prompt_then_tokens_and_training_runs(example):
    diff, losses = example.run(T=120, steps=3)
    # bf16 values all along (about eight roundings of 2^-9 between input and output, of values near the largest)
    assert diff < 2e-2
    assert len(losses) == 3 and all(l == l for l in losses)


def plain_layer(ex, layer, x, b):
    """The layer's prompt from empty caches in fp64, elementary torch operations: what autograd differentiates."""
    import torch.nn.functional as F
    L = {k: getattr(layer, k).double().requires_grad_(True)
         for k in ("norm", "norm_bias", "w_in", "w_x", "w_dt", "w_o", "taps", "conv_bias", "A_log", "skip", "dt_bias")}
    L["x"] = x.requires_grad_(True)
    T = x.shape[1]
    r = x + b
    d = r - r.mean(-1, keepdim=True)
    n = d / torch.sqrt(d.square().mean(-1, keepdim=True) + 1e-5) * L["norm"] + L["norm_bias"]
    u, z = (n @ L["w_in"]).split(ex.D, -1)
    u = F.pad(u, (0, 0, ex.K - 1, 0))
    u = F.silu(sum(u[:, i:i + T] * L["taps"][:, i] for i in range(ex.K)) + L["conv_bias"])
    low, B, C = (u @ L["w_x"]).split([ex.RANK, ex.N, ex.N], -1)
    dt = F.softplus(low @ L["w_dt"] + L["dt_bias"])
    h, ys = 0.0, []
    for t in range(T):
        a = torch.exp(-dt[:, t, :, None] * torch.exp(L["A_log"]))
        h = a * h + (dt[:, t] * u[:, t])[..., None] * B[:, t, None]
        ys.append((h * C[:, t, None]).sum(-1) + L["skip"] * u[:, t])
    return L, torch.stack(ys, 1) * F.silu(z) @ L["w_o"], r


def test_layer_gradients_equal_autograd_of_the_plain_layer(example):
    """Relative 2-norm.  About ten bf16 roundings (rms 2^-9.2 each, partly averaged out in the sums over 150 tokens) lie
    between a weight and the loss: under 1 per cent forward, a few per cent for a gradient that is itself a difference of
    larger terms: 5e-2; a missing or wrong factor would be tens of per cent."""
    layer = example.Layer(3)
    gen = torch.Generator().manual_seed(4)
    x, b, go, gr = (torch.randn(1, 150, example.WIDTH, generator=gen).to("cuda", torch.bfloat16) for _ in range(4))
    (out, r), _ = layer.prompt(x, b, layer.empty_cache(1))
    got = layer.backward(go, gr)
    L, out64, r64 = plain_layer(example, layer, x.double(), b.double())
    for have, want in ((out, out64), (r, r64)):
        assert float(((have.double() - want).norm() / want.norm()).detach()) < 2e-2
    want = torch.autograd.grad((out64 * go.double()).sum() + (r64 * gr.double()).sum(), list(L.values()))
    for name, w in zip(L, want):
        e = float((got[name].double() - w).norm() / w.norm())
        assert e < 5e-2, f"{name}: {e:.3e}"
