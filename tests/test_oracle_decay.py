"""The fp64 statement of the decayed linear attention and of the block norm: closed forms, and gradients
against central differences."""
import numpy as np
import pytest

from oracle import decay as od


def inputs(rng, B, T, Hqk, Hv, dk, dv, nseq):
    f = lambda *s: rng.normal(size=s)   # noqa: E731
    return dict(q=f(B, T, Hqk, dk), k=f(B, T, Hqk, dk), v=f(B, T, Hv, dv), g=-rng.uniform(0.01, 1.0, Hv),
                S0=f(nseq, Hv, dk, dv), do=f(B, T, Hv, dv), dS=f(nseq, Hv, dk, dv))


def test_forward_is_the_decayed_sum_over_earlier_tokens():
    rng = np.random.default_rng(1)
    x = inputs(rng, 1, 9, 1, 2, 3, 4, 1)
    out, S = od.forward(x["q"], x["k"], x["v"], x["g"], x["S0"], scale=0.5)
    for h in range(2):
        for t in range(9):
            want = np.exp(x["g"][h] * (t + 1)) * x["q"][0, t, 0] @ x["S0"][0, h]
            for j in range(t + 1):
                want = want + np.exp(x["g"][h] * (t - j)) * (x["q"][0, t, 0] @ x["k"][0, j, 0]) * x["v"][0, j, h]
            np.testing.assert_allclose(out[0, t, h], 0.5 * want, rtol=1e-12, atol=1e-12)


def test_no_decay_is_the_plain_running_sum_and_full_decay_forgets():
    rng = np.random.default_rng(2)
    x = inputs(rng, 1, 6, 1, 1, 2, 3, 1)
    _, S = od.forward(x["q"], x["k"], x["v"], np.zeros(1))
    np.testing.assert_allclose(S[0, 0], np.einsum("tk,tv->kv", x["k"][0, :, 0], x["v"][0, :, 0]), rtol=1e-12)
    _, S = od.forward(x["q"], x["k"], x["v"], np.array([-np.inf]), x["S0"])
    np.testing.assert_allclose(S[0, 0], np.outer(x["k"][0, -1, 0], x["v"][0, -1, 0]), rtol=1e-12)


def test_packed_and_steps_are_the_separate_runs():
    rng = np.random.default_rng(3)
    cu = [0, 4, 4, 5, 11]
    x = inputs(rng, 1, 11, 2, 4, 3, 5, 4)
    out, S = od.forward(x["q"], x["k"], x["v"], x["g"], x["S0"], 0.7, cu)
    for i in range(4):
        sl = slice(cu[i], cu[i + 1])
        o, s = od.forward(x["q"][:, sl], x["k"][:, sl], x["v"][:, sl], x["g"], x["S0"][i:i + 1], 0.7)
        np.testing.assert_allclose(out[:, sl], o, rtol=1e-13)
        np.testing.assert_allclose(S[i], s[0], rtol=1e-13)
    pool = x["S0"].copy()
    for t in range(5, 11):
        o, pool = od.step(x["q"][0, t][None], x["k"][0, t][None], x["v"][0, t][None], x["g"], pool, [3], 0.7)
        np.testing.assert_allclose(o[0], out[0, t], rtol=1e-12)
    np.testing.assert_allclose(pool[3], S[3], rtol=1e-12)
    o, same = od.step(x["q"][0, :1], x["k"][0, :1], x["v"][0, :1], x["g"], pool, [-1])
    assert not o.any() and np.array_equal(same, pool)


def difference(loss, a, h=1e-6):
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + h
        up = loss()
        a[i] = keep - h
        g[i] = (up - loss()) / (2 * h)
        a[i] = keep
    return g


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 7]])
def test_backward_equals_central_differences(cu):
    rng = np.random.default_rng(4)
    B, T = (2, 4) if cu is None else (1, 7)
    x = inputs(rng, B, T, 1, 2, 2, 3, B if cu is None else 3)

    def loss():
        o, S = od.forward(x["q"], x["k"], x["v"], x["g"], x["S0"], 0.6, cu)
        return (o * x["do"]).sum() + (S * x["dS"]).sum()

    got = od.backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS"], 0.6, cu)
    for name, g in zip(("q", "k", "v", "S0"), got):
        np.testing.assert_allclose(g, difference(loss, x[name]), rtol=1e-6, atol=1e-7, err_msg=name)


@pytest.mark.parametrize("cols", [None, 1, 8])
@pytest.mark.parametrize("scaled", [False, True])
def test_block_norm_backward_equals_central_differences(cols, scaled):
    rng = np.random.default_rng(5)
    f = lambda *s: rng.normal(size=s)   # noqa: E731
    x, b, wa, wb, dr, dn = f(3, 8), f(3, 8), f(8), f(8), f(3, 8), f(3, 8)
    u, c = None if cols is None else f(3, cols), f(8) if scaled else None

    def loss():
        r, n = od.block_norm(x, b, wa, wb, u, c, 1e-3)
        return (r * dr).sum() + (n * dn).sum()

    got = od.block_norm_backward(x, b, wa, wb, dr, dn, u, c, 1e-3)
    for name, g, a in zip(("x", "b", "post", "pre", "gate", "scale"), got, (x, b, wa, wb, u, c)):
        if a is None:
            assert g is None
        else:
            np.testing.assert_allclose(g, difference(loss, a), rtol=1e-6, atol=1e-7, err_msg=name)
