"""One layer with a selective state space scan as its mixer, used as a model would use it: a prompt and then token by
token, and one training step.

    x, b -> layer norm of x + b -> x | gate projection -> causal conv + SiLU -> delta | B | C projection -> delta's own
      -> selective scan with skip and gate -> output projection

The projections are plain matrix products; everything between them is the library's.  Run on a GB300 with the library
built:  python examples/scan_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_recurrence_03_gb300 as gdn   # noqa: E402

WIDTH, D, N, RANK, K = 512, 1024, 16, 32, 4   # residual stream, channels, states a channel, rank of delta, conv taps
BF16 = torch.bfloat16


class Layer:
    def __init__(self, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)

        def weight(*shape, std=None, mean=0.0, dtype=BF16):
            std = shape[0] ** -0.5 if std is None else std
            return (mean + std * torch.randn(*shape, generator=gen)).to(device=device, dtype=dtype)

        f32 = torch.float32
        self.norm, self.norm_bias = weight(WIDTH, std=0.1, mean=1.0, dtype=f32), weight(WIDTH, std=0.1, dtype=f32)
        self.w_in, self.w_x, self.w_dt = weight(WIDTH, 2 * D), weight(D, RANK + 2 * N), weight(RANK, D, std=0.1)
        self.w_o = weight(D, WIDTH)
        self.taps = weight(D, K, std=0.5, dtype=f32)
        self.conv_bias = weight(D, std=0.1, dtype=f32)
        self.A_log = torch.log(torch.arange(1.0, N + 1)).expand(D, N).contiguous().to(device)
        self.skip = weight(D, std=0.1, mean=1.0, dtype=f32)
        step = torch.exp(torch.empty(D).uniform_(-6.9, -2.3, generator=gen))   # dt of 0.001 to 0.1 at first
        self.dt_bias = (step + torch.log(-torch.expm1(-step))).to(device)

    def empty_cache(self, n):
        """The conv's last inputs and the scan's states of n sequences."""
        return torch.zeros(n, K - 1, D, dtype=BF16, device="cuda"), torch.zeros(n, D, N, device="cuda")

    def split(self, u):
        """delta, B and C of the conv's output; B and C are slices of one projection."""
        p = u @ self.w_x
        return p, p[..., :RANK] @ self.w_dt, p[..., RANK:RANK + N].unsqueeze(-2), p[..., RANK + N:].unsqueeze(-2)

    def prompt(self, x, b, cache):
        """x (residual stream) and b (the layer before's output) [B, T, WIDTH] -> (this layer's output, residual stream);
        the cache is replaced."""
        taps_in, h = cache
        n, r = gdn.gdn_layer_norm_fwd(x, self.norm, self.norm_bias, residual=b)
        xz = n @ self.w_in
        u, taps_out = gdn.gdn_causal_conv1d_fwd(xz[..., :D], self.taps, taps_in, bias=self.conv_bias)
        p, delta, B, C = self.split(u)
        y, h = gdn.gdn_selective_scan_fwd(u, delta, self.A_log, B, C, h, skip=self.skip, dt_bias=self.dt_bias, z=xz[..., D:])
        self.saved = (x, b, n, xz, u, p, delta, y)
        return (y @ self.w_o, r), (taps_out, h)

    def token(self, x, b, cache):
        """The same for one token of each sequence, [N, WIDTH]; the cache is updated in place."""
        taps, h = cache
        n, r = gdn.gdn_layer_norm_fwd(x, self.norm, self.norm_bias, residual=b)
        xz = n @ self.w_in
        u = gdn.gdn_causal_conv1d_step(xz[..., :D], self.taps, taps, bias=self.conv_bias)
        _, delta, B, C = self.split(u)
        y = gdn.gdn_selective_scan_step(u, delta, self.A_log, B, C, h, skip=self.skip, dt_bias=self.dt_bias, z=xz[..., D:])
        return y @ self.w_o, r

    def backward(self, grad_out, grad_r):
        """Gradients of the last prompt (from empty caches) by the layer's weights and its input, for dL/d(output) and
        dL/d(residual stream)."""
        x, b, n, xz, u, p, delta, y = self.saved
        rows = lambda t: t.reshape(-1, t.shape[-1])   # noqa: E731
        g = {"w_o": rows(y).T @ rows(grad_out)}
        _, _, B, C = self.split(u)
        # the gradients of the packed projections are written in place
        gp, gxz = torch.empty_like(p), torch.empty_like(xz)
        gu, gdelta, g["A_log"], _, _, g["skip"], g["dt_bias"], _, _ = gdn.gdn_selective_scan_bwd(
            u, delta, self.A_log, B, C, None, grad_out @ self.w_o.T, skip=self.skip, dt_bias=self.dt_bias, z=xz[..., D:],
            want_grad_h0=False, grads=(gp[..., RANK:RANK + N].unsqueeze(-2), gp[..., RANK + N:].unsqueeze(-2), gxz[..., D:]))
        g["w_dt"] = rows(p[..., :RANK]).T @ rows(gdelta)
        gp[..., :RANK] = gdelta @ self.w_dt.T
        g["w_x"] = rows(u).T @ rows(gp)
        gu = gu + gp @ self.w_x.T
        gx, g["taps"], _, g["conv_bias"] = gdn.gdn_causal_conv1d_bwd(xz[..., :D], self.taps, gu, bias=self.conv_bias,
                                                                     want_grad_cache_in=False)
        gxz[..., :D] = gx
        g["w_in"] = rows(n).T @ rows(gxz)
        g["x"], g["norm"], g["norm_bias"] = gdn.gdn_layer_norm_bwd(x, self.norm, gxz @ self.w_in.T, residual=b, grad_r=grad_r)
        return g


def run(T=300, steps=20, seed=0):
    """(largest difference between tokens fed one by one and the same tokens in the prompt, relative to the largest
    value; the training losses)."""
    layer = Layer(seed)
    gen = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(2, T, WIDTH, generator=gen).to("cuda", BF16)
    b = torch.randn(2, T, WIDTH, generator=gen).to("cuda", BF16)
    (whole, _), _ = layer.prompt(x, b, layer.empty_cache(2))
    (part, _), cache = layer.prompt(x[:, :T - 5].contiguous(), b[:, :T - 5].contiguous(), layer.empty_cache(2))
    got = torch.cat([part] + [layer.token(x[:, t].contiguous(), b[:, t].contiguous(), cache)[0][:, None]
                              for t in range(T - 5, T)], 1)
    diff = float((got.float() - whole.float()).abs().max() / whole.float().abs().max())

    target = torch.randn(2, T, WIDTH, generator=gen).to("cuda")
    losses = []
    for _ in range(steps):
        (out, _), _ = layer.prompt(x, b, layer.empty_cache(2))
        err = out.float() - target
        losses.append(float(err.square().mean()))
        grads = layer.backward((err / T).to(BF16), torch.zeros_like(x))
        for name, grad in grads.items():
            if name != "x":
                w = getattr(layer, name)
                w -= (0.05 * grad.float()).to(w.dtype)
    gdn.check_device_status()
    return diff, losses


if __name__ == "__main__":
    diff, losses = run()
    print(f"prompt then tokens against the whole prompt: {diff:.2e} of the largest value")
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
