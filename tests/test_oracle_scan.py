"""The fp64 statement of the selective scan and the layer norm, pinned: against sums written out, limits with a closed
form, and differences of its own forward pass."""
import numpy as np
import pytest

from oracle import scan as os_


def inputs(rng, B, T, D, G, N, nseq):
    f = lambda *s: rng.normal(size=s)   # noqa: E731
    return dict(u=f(B, T, D), delta=f(B, T, D), A_log=0.5 * f(D, N), B=f(B, T, G, N), C=f(B, T, G, N), h0=f(nseq, D, N),
                skip=f(D), dt_bias=f(D), z=f(B, T, D))


def test_forward_is_the_sum_over_earlier_tokens():
    x = inputs(np.random.default_rng(0), 2, 6, 4, 2, 3, 2)
    y, hf = os_.forward(**x)
    dt = np.log1p(np.exp(x["delta"] + x["dt_bias"]))
    A = -np.exp(x["A_log"])
    for b in range(2):
        for d in range(4):
            g = d // 2
            for t in range(6):
                total = x["skip"][d] * x["u"][b, t, d]
                for n in range(3):
                    total += x["C"][b, t, g, n] * np.exp(A[d, n] * dt[b, :t + 1, d].sum()) * x["h0"][b, d, n]
                    for s in range(t + 1):
                        decay = np.exp(A[d, n] * dt[b, s + 1:t + 1, d].sum())
                        total += x["C"][b, t, g, n] * decay * dt[b, s, d] * x["u"][b, s, d] * x["B"][b, s, g, n]
                z = x["z"][b, t, d]
                assert np.isclose(y[b, t, d], total * z / (1 + np.exp(-z)), rtol=1e-12)
    assert hf.shape == (2, 4, 3)


def test_limits():
    x = inputs(np.random.default_rng(1), 1, 5, 2, 1, 2, 1)
    x.update(skip=None, z=None, h0=None, dt_bias=None)
    dt = np.log1p(np.exp(x["delta"]))[0]
    write = dt[..., None] * x["u"][0][..., None] * x["B"][0]
    # no decay: plain sums; all decay: the last write alone
    for rate, want in ((-np.inf, write.cumsum(0)), (50.0, write)):
        x["A_log"] = np.full((2, 2), rate)
        y, hf = os_.forward(**x)
        assert np.allclose(hf[0], want[-1]) and np.allclose(y[0], (want * x["C"][0]).sum(-1))


def test_packed_is_each_sequence_alone():
    x = inputs(np.random.default_rng(2), 1, 9, 4, 2, 3, 4)
    cu = [0, 4, 4, 5, 9]
    y, hf = os_.forward(**x, cu=cu)
    g = os_.backward(x["u"], x["delta"], x["A_log"], x["B"], x["C"], x["u"], x["h0"], x["h0"], x["skip"], x["dt_bias"], x["z"], cu)
    total = 0
    for i in range(4):
        part = {k: (v[:, cu[i]:cu[i + 1]] if k in ("u", "delta", "B", "C", "z") else v) for k, v in x.items()}
        part["h0"] = x["h0"][i:i + 1]
        yi, hi = os_.forward(**part)
        assert np.allclose(yi, y[:, cu[i]:cu[i + 1]]) and np.allclose(hi[0], hf[i])
        gi = os_.backward(part["u"], part["delta"], x["A_log"], part["B"], part["C"], part["u"], part["h0"], part["h0"],
                          x["skip"], x["dt_bias"], part["z"])
        assert np.allclose(gi[0], g[0][:, cu[i]:cu[i + 1]]) and np.allclose(gi[8][0], g[8][i])
        total = total + gi[2]
    assert np.allclose(total, g[2])


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 7]])
def test_backward_equals_differences(cu):
    nseq = 2 if cu is None else 3
    x = inputs(np.random.default_rng(3), 2 if cu is None else 1, 5 if cu is None else 7, 4, 2, 3, nseq)
    rng = np.random.default_rng(4)
    gy, gh = rng.normal(size=x["u"].shape), rng.normal(size=x["h0"].shape)
    names = ("u", "delta", "A_log", "B", "C", "skip", "dt_bias", "z", "h0")
    grads = os_.backward(x["u"], x["delta"], x["A_log"], x["B"], x["C"], gy, x["h0"], gh, x["skip"], x["dt_bias"], x["z"], cu)

    def loss(v):
        y, h = os_.forward(**v, cu=cu)
        return (y * gy).sum() + (h * gh).sum()

    for name, g in zip(names, grads):
        d = rng.normal(size=x[name].shape)
        up, down = ({**x, name: x[name] + s * 1e-6 * d} for s in (1, -1))
        assert np.isclose((loss(up) - loss(down)) / 2e-6, (g * d).sum(), rtol=1e-6, atol=1e-7), name


def test_step_is_a_prompt_of_one_token():
    x = inputs(np.random.default_rng(5), 3, 1, 4, 1, 2, 3)
    y, h = os_.forward(**x)
    row = {k: (v[:, 0] if k in ("u", "delta", "B", "C", "z") else v) for k, v in x.items() if k != "h0"}
    ys, hs = os_.step(**row, h=x["h0"])
    assert np.allclose(ys, y[:, 0]) and np.allclose(hs, h)
    pool = np.concatenate([x["h0"], x["h0"]])
    ys, hs = os_.step(**row, h=pool, slots=[4, -1, 0])
    assert np.allclose(hs[4], os_.step(**row, h=x["h0"][[1, 1, 1]])[1][0]) and not ys[1].any()
    assert np.array_equal(hs[[1, 2, 3, 5]], pool[[1, 2, 3, 5]])


def test_layer_norm_and_its_gradients():
    rng = np.random.default_rng(6)
    f = lambda *s: rng.normal(size=s)   # noqa: E731
    x, b, w, bias, gn, gr = f(3, 7), f(3, 7), f(7), f(7), f(3, 7), f(3, 7)
    n, r = os_.layer_norm(x, w, bias, b)
    assert np.array_equal(r, x + b)
    rh = (n - bias) / w
    assert np.allclose(rh.mean(-1), 0) and np.allclose((rh ** 2).mean(-1), 1, atol=1e-4)
    dx, dw, db = os_.layer_norm_backward(x, w, gn, b, gr)
    loss = lambda x, w, bias: sum((t * g).sum() for t, g in zip(os_.layer_norm(x, w, bias, b), (gn, gr)))   # noqa: E731
    for i, (v, g) in enumerate(((x, dx), (w, dw), (bias, db))):
        d = f(*v.shape)
        up, down = ([a + s * 1e-6 * d if j == i else a for j, a in enumerate((x, w, bias))] for s in (1, -1))
        assert np.isclose((loss(*up) - loss(*down)) / 2e-6, (g * d).sum(), rtol=1e-6, atol=1e-7)
