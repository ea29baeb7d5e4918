"""GPU: the causal convolution with a bias (prompt, token step, their q | k | v forms, gradients) against the fp64 oracle.

Tolerances, of the largest value of the tensor.  fp32 outputs: u is at most five rounded terms (5 x 2^-24 of a sum of
magnitudes that is about twice the largest output), SiLU by an exponential and a division of about 2^-21 each: 2^-18.
bf16 outputs: half a step, 2^-8, and the 2^-11 of the tanh that SiLU takes then, on half the value: 2^-8 + 2^-11.
Gradients are fp32: du = dy (s + u s (1 - s)) is off by about 2^-20 of its largest value (s by 2^-21, u as above, and the
terms cancel where the slope is zero), an input's gradient adds four of them: 2^-17.  The sums over at most 512 tokens:
chains of at most 64 terms and ten joins, 74 x 2^-24 of sum |du| (largest du times 512) against a largest sum of no less
than a tenth of that over the channels: below 2^-14; each du's own 2^-20 adds 10 x 2^-20: 2^-14 + 2^-16 in all."""
import numpy as np
import pytest

import gdn_inputs as gi
from oracle import conv as oconv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from gpu_util import rel_err, up  # noqa: E402
import gated_deltanet_recurrence_03_gb300 as gdn  # noqa: E402

TOL_Y = {"f32": 2.0 ** -18, "bf16": 2.0 ** -8 + 2.0 ** -11}
TOL_X, TOL_SUM = 2.0 ** -17, 2.0 ** -14 + 2.0 ** -16
F32 = torch.float32
SPANS = {"batch": None, "one token": (1,), "packed": (0, 1, 2, 65, 0, 130, 3)}


def case(seed, spans, C, K, dtype):
    lens = SPANS[spans]
    lead = (3, 150) if lens is None else (1, sum(lens))
    nseq, n = (3 if lens is None else len(lens)), lead[0] * lead[1] * C
    cu = None if lens is None else np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    r = lambda i, *s: gi.normals(seed, i, int(np.prod(s))).reshape(*s)   # noqa: E731
    d = dict(x=gi.round_to_dtype(r(0, *lead, C), dtype), w=gi.round_to_dtype(0.5 * r(1, C, K), "f32"),
             cache=gi.round_to_dtype(r(2, nseq, K - 1, C), dtype), dy=gi.round_to_dtype(r(3, *lead, C), dtype),
             dco=gi.round_to_dtype(r(4, nseq, K - 1, C), dtype), bias=gi.round_to_dtype(r(5, C), "f32"))
    assert n == d["x"].size
    return d, cu, None if cu is None else torch.from_numpy(cu).cuda()


def backward(d, cut, dtype, bias, **kw):
    return gdn.gdn_causal_conv1d_bwd(up(d["x"], dtype), up(d["w"], F32), up(d["dy"], dtype), up(d["cache"], dtype), bias=bias,
                                     grad_cache_out=up(d["dco"], dtype), cu_seqlens=cut, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("spans", list(SPANS))
def test_prompt(spans, K, dtype):
    d, cu, cut = case(80 + K, spans, 96, K, dtype)
    y, co = gdn.gdn_causal_conv1d_fwd(up(d["x"], dtype), up(d["w"], F32), up(d["cache"], dtype), bias=up(d["bias"], F32),
                                      cu_seqlens=cut)
    ry, rc = oconv.causal_conv1d(d["x"], d["w"], d["cache"], cu_seqlens=cu, bias=d["bias"])
    assert rel_err(ry, y.float().cpu().numpy()) <= TOL_Y[dtype]
    np.testing.assert_array_equal(co.float().cpu().numpy(), rc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("spans", list(SPANS))
def test_gradients(spans, K, dtype):
    d, cu, cut = case(90 + K, spans, 200, K, dtype)   # 200 channels: the last block of channels is ragged
    got = backward(d, cut, dtype, up(d["bias"], F32))
    want = oconv.causal_conv1d_backward(d["x"], d["w"], d["dy"], d["cache"], cu_seqlens=cu, dcache_out=d["dco"],
                                        bias=d["bias"])
    for name, tol, have, ref in zip(("x", "w", "cache", "bias"), (TOL_X, TOL_SUM, TOL_X, TOL_SUM), got, want):
        if ref.size and have is not None:
            assert rel_err(ref, have.cpu().numpy()) <= tol, name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 4])
def test_tokens_one_by_one_are_the_prompt(K, dtype):
    d, _, _ = case(100, "batch", 72, K, dtype)
    x, w, bias, cache = up(d["x"], dtype), up(d["w"], F32), up(d["bias"], F32), up(d["cache"], dtype)
    want, last = gdn.gdn_causal_conv1d_fwd(x, w, cache, bias=bias)
    for t in range(20):
        y = gdn.gdn_causal_conv1d_step(x[:, t], w, cache, bias=bias)
        assert torch.equal(y, want[:, t])
    for t in range(20, x.shape[1]):
        gdn.gdn_causal_conv1d_step(x[:, t], w, cache, bias=bias)
    assert torch.equal(cache, last)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_qkv_forms_are_the_split(dtype):
    d, _, cut = case(101, "packed", 128, 4, dtype)
    x, w, bias, cache = up(d["x"], dtype), up(d["w"], F32), up(d["bias"], F32), up(d["cache"], dtype)
    widths = (32, 40, 56)
    y, co = gdn.gdn_causal_conv1d_fwd(x, w, cache, bias=bias, cu_seqlens=cut)
    *parts, co2 = gdn.gdn_causal_conv1d_fwd_qkv(x, w, widths, cache, bias=bias, cu_seqlens=cut)
    parts = parts[0] if len(parts) == 1 else parts
    assert torch.equal(torch.cat(list(parts), -1), y) and torch.equal(co, co2)
    rows, c1, c2 = x[0, :7], cache.clone(), cache.clone()
    y = gdn.gdn_causal_conv1d_step(rows, w, c1, bias=bias)
    parts = gdn.gdn_causal_conv1d_step_qkv(rows, w, c2, widths, bias=bias)
    assert torch.equal(torch.cat(list(parts), -1), y) and torch.equal(c1, c2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_bias_of_zeros_is_none(dtype):
    """0 + w x is w x: every result is the same bit for bit (but for the sign of a zero)."""
    d, _, cut = case(102, "packed", 136, 4, dtype)
    zero = torch.zeros(136, device="cuda")
    args = up(d["x"], dtype), up(d["w"], F32), up(d["cache"], dtype)
    for a, b in zip(gdn.gdn_causal_conv1d_fwd(*args, bias=zero, cu_seqlens=cut), gdn.gdn_causal_conv1d_fwd(*args, cu_seqlens=cut)):
        assert torch.equal(a, b)
    got, plain = backward(d, cut, dtype, zero), backward(d, cut, dtype, None)
    assert len(got) == 4 and len(plain) == 3
    for a, b in zip(got, plain):
        assert torch.equal(a, b)


def test_misaligned_rows_of_weights_and_bias():
    d, cu, cut = case(103, "packed", 64, 4, "bf16")
    odd = lambda a: torch.cat([torch.zeros(1), torch.from_numpy(a.astype(np.float32)).flatten()]).cuda()[1:].view(a.shape)   # noqa: E731
    y, _ = gdn.gdn_causal_conv1d_fwd(up(d["x"], "bf16"), odd(d["w"]), up(d["cache"], "bf16"), bias=odd(d["bias"]), cu_seqlens=cut)
    y2, _ = gdn.gdn_causal_conv1d_fwd(up(d["x"], "bf16"), up(d["w"], F32), up(d["cache"], "bf16"), bias=up(d["bias"], F32),
                                      cu_seqlens=cut)
    assert torch.equal(y, y2)
    for a, b in zip(backward(d, cut, "bf16", odd(d["bias"])), backward(d, cut, "bf16", up(d["bias"], F32))):
        assert torch.equal(a, b)


def test_left_out_gradients_and_an_empty_batch():
    d, _, cut = case(104, "packed", 64, 4, "bf16")
    bias = up(d["bias"], F32)
    full = backward(d, cut, "bf16", bias)
    part = backward(d, cut, "bf16", bias, want_grad_w=False, want_grad_cache_in=False)
    assert part[1] is None and part[2] is None and torch.equal(part[0], full[0]) and torch.equal(part[3], full[3])
    x = torch.zeros(0, 5, 64, device="cuda", dtype=torch.bfloat16)
    gx, _, _, gb = gdn.gdn_causal_conv1d_bwd(x, up(d["w"], F32), x, bias=bias)
    assert gx.shape == x.shape and torch.equal(gb, torch.zeros(64, device="cuda"))


def test_captured_and_replayed_with_other_values():
    d, _, cut = case(105, "packed", 64, 4, "bf16")
    bias = up(d["bias"], F32)
    x, w, dy = up(d["x"], "bf16"), up(d["w"], F32), up(d["dy"], "bf16")
    run = lambda: (gdn.gdn_causal_conv1d_fwd(x, w, bias=bias, cu_seqlens=cut)[0],   # noqa: E731
                   *gdn.gdn_causal_conv1d_bwd(x, w, dy, bias=bias, cu_seqlens=cut, want_grad_cache_in=False)[::3])
    run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = run()
    for scale in (1.0, -0.5):
        bias.mul_(scale)
        x.mul_(scale)
        graph.replay()
        for a, b in zip(out, run()):
            assert torch.equal(a, b)
