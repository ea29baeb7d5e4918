"""One layer with a decaying linear attention as its mixer, used as a model would use it: a prompt and then token
by token, and one training step.

    n -> q | k | v projection -> causal conv + SiLU -> linear attention with a decay per head -> output gate
      -> output projection -> norm, gate, residual scale and residual -> norm for the next layer

The projections are plain matrix products; everything between them is the library's.  Run on a GB300 with the
library built:  python examples/decay_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_recurrence_03_gb300 as gdn   # noqa: E402

D, HQK, HV, HEAD, K = 512, 2, 4, 128, 4            # width, query/key heads, value heads, head dim, conv taps
WIDTHS = (HQK * HEAD, HQK * HEAD, HV * HEAD)       # of q, k and v in the packed projection
BF16 = torch.bfloat16


class Layer:
    def __init__(self, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)

        def weight(*shape, std=None, mean=0.0, dtype=BF16):
            std = shape[0] ** -0.5 if std is None else std
            return (mean + std * torch.randn(*shape, generator=gen)).to(device=device, dtype=dtype)

        f32 = torch.float32
        self.w_qkv, self.w_z, self.w_u = weight(D, sum(WIDTHS)), weight(D, HV * HEAD), weight(D, D)
        self.w_o = weight(HV * HEAD, D)
        self.taps = weight(sum(WIDTHS), K, std=0.5, dtype=f32)
        self.head_norm = weight(HEAD, std=0.1, mean=1.0, dtype=f32)
        self.post, self.pre = weight(D, std=0.1, mean=1.0, dtype=f32), weight(D, std=0.1, mean=1.0, dtype=f32)
        self.res_scale = weight(D, std=0.1, mean=0.5, dtype=f32)
        # memories from a few tokens to hundreds, a constant of each head
        self.log_decay = -torch.exp2(-torch.linspace(2.0, 8.0, HV)).to(device)
        self.scale = HEAD ** -0.5

    def empty_cache(self, n):
        """The conv's last inputs and the attention's states of n sequences."""
        return (torch.zeros(n, K - 1, sum(WIDTHS), dtype=BF16, device="cuda"),
                torch.zeros(n, HV, HEAD, HEAD, device="cuda"))

    def prompt(self, x, n, cache):
        """x (residual stream) and n (its norm) [B, T, D] -> (x, n) of the next layer; the cache is replaced."""
        B, T, _ = x.shape
        taps_in, S = cache
        p = n @ self.w_qkv
        (q, k, v), taps_out = gdn.gdn_causal_conv1d_fwd_qkv(p, self.taps, WIDTHS, taps_in)
        q, k, v = q.view(B, T, HQK, HEAD), k.view(B, T, HQK, HEAD), v.view(B, T, HV, HEAD)
        o, S = gdn.gdn_decay_attn_fwd(q, k, v, self.log_decay, S, scale=self.scale)
        z = (n @ self.w_z).view(B, T, HV, HEAD)
        y = gdn.gdn_output_gate_fwd(o, z, self.head_norm)
        b, u = y.view(B, T, HV * HEAD) @ self.w_o, n @ self.w_u
        self.saved = (x, n, p, q, k, v, o, z, y, b, u)
        return gdn.gdn_block_norm_fwd(x, b, self.post, self.pre, gate=u, res_scale=self.res_scale), (taps_out, S)

    def token(self, x, n, cache):
        """The same for one token of each sequence, [N, D]; the cache is updated in place."""
        taps, S = cache
        q, k, v = gdn.gdn_causal_conv1d_step_qkv(n @ self.w_qkv, self.taps, taps, WIDTHS)
        N = x.shape[0]
        o = gdn.gdn_decay_attn_step(q.view(N, HQK, HEAD), k.view(N, HQK, HEAD), v.view(N, HV, HEAD), self.log_decay, S,
                                    scale=self.scale)
        y = gdn.gdn_output_gate_fwd(o, (n @ self.w_z).view(N, HV, HEAD), self.head_norm)
        return gdn.gdn_block_norm_fwd(x, y.view(N, HV * HEAD) @ self.w_o, self.post, self.pre, gate=n @ self.w_u,
                                      res_scale=self.res_scale)

    def backward(self, grad_x, grad_n):
        """Gradients of the last prompt (from empty caches) by the layer's weights, for dL/dx, dL/dn of its outputs."""
        x, n, p, q, k, v, o, z, y, b, u = self.saved
        B, T, _ = x.shape
        g = {}
        gx, gb, g["post"], g["pre"], gu, g["res_scale"] = gdn.gdn_block_norm_bwd(
            x, b, self.post, self.pre, grad_x, grad_n, gate=u, res_scale=self.res_scale)
        rows = lambda t: t.reshape(B * T, -1)   # noqa: E731
        g["w_o"], g["w_u"] = rows(y).T @ rows(gb), rows(n).T @ rows(gu)
        gy = (gb @ self.w_o.T).view(B, T, HV, HEAD)
        go, gz, g["head_norm"] = gdn.gdn_output_gate_bwd(o, z, self.head_norm, gy)
        g["w_z"] = rows(n).T @ rows(gz.to(BF16))
        # the three gradients side by side, as the conv's backward takes them
        packed = torch.empty(B, T, sum(WIDTHS), dtype=BF16, device=x.device)
        views = [t.unflatten(-1, (h, HEAD)) for t, h in zip(packed.split(WIDTHS, -1), (HQK, HQK, HV))]
        gdn.gdn_decay_attn_bwd(q, k, v, self.log_decay, None, go.to(BF16), scale=self.scale, want_grad_S0=False,
                               grads=views)
        gp, g["taps"], _ = gdn.gdn_causal_conv1d_bwd(p, self.taps, packed, want_grad_cache_in=False)
        g["w_qkv"] = rows(n).T @ rows(gp.to(BF16))
        return g


def run(T=300, steps=20, seed=0):
    """(largest difference between tokens fed one by one and the same tokens in the prompt, relative to the largest
    value; the training losses)."""
    layer = Layer(seed)
    gen = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(2, T, D, generator=gen).to("cuda", BF16)
    n = torch.randn(2, T, D, generator=gen).to("cuda", BF16)
    (whole, _), _ = layer.prompt(x, n, layer.empty_cache(2))
    (part, _), cache = layer.prompt(x[:, :T - 5].contiguous(), n[:, :T - 5].contiguous(), layer.empty_cache(2))
    got = torch.cat([part] + [layer.token(x[:, t].contiguous(), n[:, t].contiguous(), cache)[0][:, None]
                              for t in range(T - 5, T)], 1)
    diff = float((got.float() - whole.float()).abs().max() / whole.float().abs().max())

    target = torch.randn(2, T, D, generator=gen).to("cuda")
    losses = []
    for _ in range(steps):
        (_, out), _ = layer.prompt(x, n, layer.empty_cache(2))
        err = out.float() - target
        losses.append(float(err.square().mean()))
        grads = layer.backward(torch.zeros_like(x), (err / T).to(BF16))
        for name, grad in grads.items():
            w = getattr(layer, name)
            w -= (0.05 * grad.float()).to(w.dtype)
    gdn.check_device_status()
    return diff, losses


if __name__ == "__main__":
    diff, losses = run()
    print(f"prompt then tokens against the whole prompt: {diff:.2e} of the largest value")
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
