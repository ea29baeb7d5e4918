"""GPU: the layer norm with its residual add, and its gradients, against oracle.scan's fp64 statement.

Tolerances (max error over max value).  fp32: two row sums of D values in fp32 and a reciprocal root good to a few 2^-23:
1e-5.  bf16 results: one rounding, 2^-9 of the value: 2^-8.  Weight gradients are fp32 sums over the rows of fp32 values,
whatever the inputs' type: 1e-5."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import scan as os_   # noqa: E402

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 1e-5, "bf16": 2.0 ** -8}


def gdn():
    import gated_deltanet_recurrence_03_gb300 as g
    return g


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def close(want, got, tol, what):
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if want.size:
        err = np.abs(got - want).max() / max(np.abs(want).max(), 1e-30)
        assert err <= tol, f"{what}: {err:.3e} > {tol:.1e}"


def make(dtype, rows, D, residual=True, bias=True, gr=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    d = lambda *s: n(*s).to(DT[dtype]).cuda()   # noqa: E731
    return dict(x=d(rows, D), residual=d(rows, D) if residual else None, w=(1 + 0.1 * n(D)).cuda(),
                bias=n(D).cuda() if bias else None, gn=d(rows, D), gr=d(rows, D) if gr else None)


CASES = [(dtype, rows, D, *opt)
         for dtype in ("f32", "bf16")
         for rows, D, opt in ((1, 8, (True, True, True)), (3, 136, (False, True, False)), (1, 2048, (True, False, False)),
                              (700, 1160, (True, True, True)), (37, 4096, (False, False, True)),
                              (5, 4104, (True, True, False)), (1300, 264, (False, True, True)),
                              (2, 8192, (True, True, True)), (333, 5008, (True, True, True)),
                              (4000, 64, (False, True, False)), (6000, 256, (True, True, True)))]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(case):
    x = make(*case)
    tol = TOL[case[0]]
    n, r = gdn().gdn_layer_norm_fwd(x["x"], x["w"], x["bias"], residual=x["residual"])
    nw, rw = os_.layer_norm(f64(x["x"]), f64(x["w"]), f64(x["bias"]), f64(x["residual"]))
    close(nw, n, tol, "n")
    if x["residual"] is None:
        assert r is None
    else:
        close(rw, r, tol, "r")
    got = gdn().gdn_layer_norm_bwd(x["x"], x["w"], x["gn"], residual=x["residual"], grad_r=x["gr"])
    want = os_.layer_norm_backward(f64(x["x"]), f64(x["w"]), f64(x["gn"]), f64(x["residual"]), f64(x["gr"]))
    for name, w, g in zip(("grad_x", "grad_weight", "grad_bias"), want, got):
        close(w, g, 1e-5 if g.dtype == torch.float32 else tol, name)
    again = gdn().gdn_layer_norm_bwd(x["x"], x["w"], x["gn"], residual=x["residual"], grad_r=x["gr"])
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert gdn().gdn_layer_norm_bwd(x["x"], x["w"], x["gn"], residual=x["residual"], grad_r=x["gr"], want_grad_bias=False)[2] is None


def test_backward_equals_differences():
    """fp32, a direction at a time: the loss's curvature times the step squared and rounding over the step both stay
    below 2e-3 of the terms' size."""
    x = make("f32", 6, 64, seed=1)
    grads = gdn().gdn_layer_norm_bwd(x["x"], x["w"], x["gn"], residual=x["residual"], grad_r=x["gr"])
    gen = torch.Generator().manual_seed(2)

    def loss(v):
        n, r = gdn().gdn_layer_norm_fwd(v["x"], v["w"], v["bias"], residual=v["residual"])
        return float((n.double() * x["gn"].double()).sum() + (r.double() * x["gr"].double()).sum())

    for name, g in zip(("x", "residual", "w", "bias"), (grads[0], grads[0], grads[1], grads[2])):
        d = torch.randn(x[name].shape, generator=gen).cuda()
        h = 1e-2
        up, down = ({**x, name: x[name] + s * h * d} for s in (1, -1))
        num, ana = (loss(up) - loss(down)) / (2 * h), float((g.double() * d.double()).sum())
        size = float((g.double().abs() * d.double().abs()).sum())
        assert abs(num - ana) <= 2e-3 * size, (name, num, ana)


def test_rows_far_from_zero():
    """A mean of 1000 deviations: the sum of a row passes about 14 additions a value, each off by at most 2^-24 of the sum,
    so the mean and every deviation from it are good to 16 x 1000 2^-24."""
    gen = torch.Generator().manual_seed(3)
    x = (1000 + torch.randn(40, 1024, generator=gen)).cuda()
    w = torch.ones(1024).cuda()
    n, _ = gdn().gdn_layer_norm_fwd(x, w)
    want, _ = os_.layer_norm(f64(x), f64(w))
    assert np.abs(f64(n) - want).max() <= 16 * 1000 * 2.0 ** -24
    gn = torch.randn(40, 1024, generator=gen).cuda()
    gx, gw, gb = gdn().gdn_layer_norm_bwd(x, w, gn)
    wx, ww, wb = os_.layer_norm_backward(f64(x), f64(w), f64(gn))
    for a, b, s in ((wx, gx, 8), (ww, gw, 40), (wb, gb, 40)):
        assert np.abs(f64(b) - a).max() <= s * 16 * 1000 * 2.0 ** -24


def test_in_place_strange_rows_and_streams():
    x = make("bf16", 9, 512, seed=3)
    want = gdn().gdn_layer_norm_fwd(x["x"], x["w"], x["bias"], residual=x["residual"])
    side = torch.cuda.Stream()
    xs, bs = x["x"].clone(), x["residual"].clone()
    side.wait_stream(torch.cuda.current_stream())
    n, r = gdn().gdn_layer_norm_fwd(xs, x["w"], x["bias"], residual=bs, out=(bs, xs), stream=side)
    side.synchronize()
    assert r is xs and n is bs and torch.equal(want[0], n) and torch.equal(want[1], r)
    # rows of zeros, of one value, a NaN, an infinity: they stay in their rows
    x["x"][2], x["residual"][2], x["x"][3], x["residual"][3] = 0, 0, 5.0, 1.0
    x["x"][4, 7], x["x"][6, 100] = float("nan"), float("inf")
    n, r = gdn().gdn_layer_norm_fwd(x["x"], x["w"], x["bias"], residual=x["residual"])
    keep = [0, 1, 2, 3, 5, 7, 8]
    nw, rw = os_.layer_norm(f64(x["x"])[keep], f64(x["w"]), f64(x["bias"]), f64(x["residual"])[keep])
    close(nw, n[keep], TOL["bf16"], "n")
    close(rw, r[keep], TOL["bf16"], "r")
    assert torch.isnan(n[4]).all() and torch.isnan(n[6]).all()
    gx, _, gb = gdn().gdn_layer_norm_bwd(x["x"], x["w"], x["gn"], residual=x["residual"], grad_r=x["gr"])
    assert torch.isfinite(gx[keep]).all() and torch.isfinite(gb).all()


def test_in_a_graph():
    x = make("bf16", 333, 264, seed=4)
    f = lambda: (*gdn().gdn_layer_norm_fwd(x["x"], x["w"], x["bias"], residual=x["residual"]),   # noqa: E731
                 *gdn().gdn_layer_norm_bwd(x["x"], x["w"], x["gn"], residual=x["residual"], grad_r=x["gr"]))
    want = [t.clone() for t in f()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_no_rows_and_refusals():
    x = make("f32", 0, 64)
    n, r = gdn().gdn_layer_norm_fwd(x["x"], x["w"], x["bias"], residual=x["residual"])
    assert n.shape == r.shape == (0, 64)
    gx, gw, gb = gdn().gdn_layer_norm_bwd(x["x"], x["w"], x["gn"], residual=x["residual"], grad_r=x["gr"])
    assert gx.shape == (0, 64) and not gw.any() and not gb.any()
    x = make("f32", 4, 64)
    for bad in (dict(residual=x["gn"][:, :32]), dict(residual=x["gn"].bfloat16()), dict(x=x["x"].t().contiguous().t()),
                dict(weight=x["w"].bfloat16()), dict(bias=x["bias"][:8]), dict(out=(x["x"], None)), dict(x=x["x"].double()),
                dict(residual=x["gn"].cpu())):
        a = dict(x=x["x"], weight=x["w"], bias=x["bias"], residual=x["residual"]) | bad
        with pytest.raises((ValueError, TypeError)):
            gdn().gdn_layer_norm_fwd(**a)
    for D in (12, 8200):
        y = make("f32", 1, D)
        with pytest.raises(gdn().GdnError):
            gdn().gdn_layer_norm_fwd(y["x"], y["w"])
    with pytest.raises(gdn().GdnError):
        gdn().gdn_layer_norm_fwd(x["x"], x["w"], eps=-1.0)
    with pytest.raises(gdn().GdnError):
        gdn().gdn_layer_norm_fwd(x["x"], x["w"], residual=x["residual"], out=(x["gn"], x["gn"]))
