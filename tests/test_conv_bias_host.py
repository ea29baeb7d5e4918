"""The causal convolution's bias without a GPU: the oracle against finite differences, and what the C ABI and the binding
refuse."""
import numpy as np
import pytest

from oracle import conv
from test_abi_host import FAKE, lib, opts  # noqa: F401
from test_oracle_conv import _fd
import gated_deltanet_recurrence_03_gb300._lib as pkg_lib


@pytest.mark.parametrize("lens,K", [((4, 0, 1, 5), 4), ((7,), 2), ((5,), 1)])
def test_oracle_gradients_match_finite_differences(lens, K):
    rng = np.random.default_rng(12)
    T, C, cu = sum(lens), 3, np.concatenate([[0], np.cumsum(lens)])
    x, w, bias = rng.normal(size=(1, T, C)), rng.normal(size=(C, K)), rng.normal(size=C)
    cache, dy = rng.normal(size=(len(lens), K - 1, C)), rng.normal(size=(1, T, C))

    def loss(xx=x, ww=w, cc=cache, bb=bias):
        return float(np.sum(conv.causal_conv1d(xx, ww, cc, cu_seqlens=cu, bias=bb)[0] * dy))

    dx, dw, dc, db = conv.causal_conv1d_backward(x, w, dy, cache, cu_seqlens=cu, bias=bias)
    pairs = [(dx, _fd(lambda t: loss(xx=t), x)), (dw, _fd(lambda t: loss(ww=t), w)), (db, _fd(lambda t: loss(bb=t), bias))]
    if K > 1:
        pairs.append((dc, _fd(lambda t: loss(cc=t), cache)))
    for have, want in pairs:
        np.testing.assert_allclose(have, want, rtol=1e-6, atol=1e-8)


def test_oracle_matches_numpy_convolve_with_a_bias():
    rng = np.random.default_rng(13)
    x, w, bias = rng.normal(size=(2, 9, 4)), rng.normal(size=(4, 3)), rng.normal(size=4)
    u = np.stack([np.convolve(x[b, :, c], w[c, ::-1])[:9] for b in range(2) for c in range(4)]).reshape(2, 4, 9)
    u = u.transpose(0, 2, 1) + bias
    np.testing.assert_allclose(conv.causal_conv1d(x, w, bias=bias)[0], u / (1 + np.exp(-u)), rtol=1e-12, atol=1e-14)


def bwd(lib, ptrs=None, B=1, T=8, C=64, K=4, **kw):   # noqa: F811
    # x, w, cache_in, grad_y, grad_cache_out, grad_x, grad_w, grad_cache_in
    p = [FAKE, FAKE, 0, FAKE, 0, FAKE, FAKE, 0] if ptrs is None else ptrs
    return lib.gdn_causal_conv1d_bwd(p[0], 0, *p[1:], B, T, C, K, opts(lib, **kw))


def test_misaligned_biases_are_refused(lib):   # noqa: F811
    o = dict(conv_bias=FAKE + 2)
    bad = pkg_lib.GDN_ERR_INVALID_ARG
    assert lib.gdn_causal_conv1d_fwd(FAKE, 0, FAKE, 0, FAKE, 0, 1, 8, 64, 4, opts(lib, **o)) == bad
    assert lib.gdn_causal_conv1d_step(FAKE, 0, FAKE, FAKE, FAKE, 4, 64, 4, opts(lib, **o)) == bad
    assert lib.gdn_causal_conv1d_fwd_qkv(FAKE, 0, FAKE, 0, FAKE, FAKE, FAKE, 0, 1, 8, 64, 64, 64, 4, opts(lib, **o)) == bad
    assert lib.gdn_causal_conv1d_step_qkv(FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 64, 64, 4, opts(lib, **o)) == bad
    big = dict(workspace=FAKE, workspace_bytes=1 << 30)
    assert bwd(lib, **o, **big) == bad
    assert bwd(lib, conv_bias=FAKE, grad_conv_bias=FAKE + 2, **big) == bad


def test_gradient_of_a_bias_needs_the_bias(lib):   # noqa: F811
    assert bwd(lib, grad_conv_bias=FAKE, workspace=FAKE, workspace_bytes=1 << 30) == pkg_lib.GDN_ERR_INVALID_ARG


def test_workspace_counts_the_bias(lib):   # noqa: F811
    size = lib.gdn_causal_conv1d_bwd_workspace_size
    plain, with_bias = size(2, 100, 64, 4, opts(lib)), size(2, 100, 64, 4, opts(lib, conv_bias=FAKE, grad_conv_bias=FAKE))
    assert plain == size(2, 100, 64, 4, opts(lib, conv_bias=FAKE))   # a bias without its gradient needs no more
    assert with_bias * 4 == plain * 5                                 # four taps and the bias a channel
    short = dict(conv_bias=FAKE, grad_conv_bias=FAKE, workspace=FAKE, workspace_bytes=with_bias - 1)
    assert bwd(lib, B=2, T=100, **short) == pkg_lib.GDN_ERR_WORKSPACE
    # the bias's gradient alone, without the taps', needs it too
    p = [FAKE, FAKE, 0, FAKE, 0, FAKE, 0, 0]
    assert bwd(lib, p, conv_bias=FAKE, grad_conv_bias=FAKE) == pkg_lib.GDN_ERR_WORKSPACE


@pytest.mark.parametrize("bad", ["length", "dtype", "stride"])
def test_binding_checks_the_bias(bad):
    torch = pytest.importorskip("torch")
    from gated_deltanet_recurrence_03_gb300 import api
    bias = {"length": torch.zeros(63), "dtype": torch.zeros(64, dtype=torch.bfloat16), "stride": torch.zeros(128)[::2]}[bad]
    with pytest.raises((ValueError, TypeError)):
        api._conv_bias(None, bias, 64, bias.device)
