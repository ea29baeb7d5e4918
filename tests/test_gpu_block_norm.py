"""GPU: the norms, gate, residual scale and residual around a block in one pass, and its gradients, against
oracle.decay's fp64 statement.

Tolerances (max error over max value).  fp32: row sums of D values in fp32 and elementwise functions good to a
few 2^-23: 1e-5.  bf16 results: one rounding, 2^-9 of the value: 2^-8.  Weight gradients are fp32 sums over the
rows of fp32 values, whatever the inputs' type: 1e-5."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import decay as od   # noqa: E402

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
    err = np.abs(got - want).max() / max(np.abs(want).max(), 1e-30)
    assert err <= tol, f"{what}: {err:.3e} > {tol:.1e}"


def make(dtype, rows, D, cols, scaled, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    d = lambda *s: n(*s).to(DT[dtype]).cuda()   # noqa: E731
    return dict(x=d(rows, D), b=(3 * n(rows, D)).to(DT[dtype]).cuda(), wa=(1 + 0.1 * n(D)).cuda(), wb=(1 + 0.1 * n(D)).cuda(),
                gate={0: None, 1: d(rows, 1), 2: d(rows, D)}[cols], c=(0.5 + 0.1 * n(D)).cuda() if scaled else None,
                gr=d(rows, D), gn=d(rows, D))


CASES = [(dtype, rows, D, cols, scaled)
         for dtype in ("f32", "bf16")
         for rows, D, cols, scaled in ((1, 8, 2, True), (3, 136, 1, False), (1, 2048, 0, False), (700, 1160, 2, True),
                                       (37, 4096, 2, False), (5, 4104, 1, True), (1300, 264, 0, True), (2, 8192, 2, True), (333, 5008, 1, True), (4000, 64, 2, False))]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(case):
    x = make(*case)
    tol = TOL[case[0]]
    args = [f64(x[n]) for n in ("x", "b", "wa", "wb")]
    r, n = gdn().gdn_block_norm_fwd(x["x"], x["b"], x["wa"], x["wb"], gate=x["gate"], res_scale=x["c"], eps=1e-5)
    rw, nw = od.block_norm(*args, f64(x["gate"]), f64(x["c"]), 1e-5)
    close(rw, r, tol, "r")
    close(nw, n, tol, "n")
    got = gdn().gdn_block_norm_bwd(x["x"], x["b"], x["wa"], x["wb"], x["gr"], x["gn"], gate=x["gate"], res_scale=x["c"],
                                   eps=1e-5)
    want = od.block_norm_backward(*args, f64(x["gr"]), f64(x["gn"]), f64(x["gate"]), f64(x["c"]), 1e-5)
    for name, w, g in zip(("grad_x", "grad_b", "grad_post", "grad_pre", "grad_gate", "grad_scale"), want, got):
        if w is None:
            assert g is None, name
        else:
            close(w, g, 1e-5 if g.dtype == torch.float32 else tol, name)
    again = gdn().gdn_block_norm_bwd(x["x"], x["b"], x["wa"], x["wb"], x["gr"], x["gn"], gate=x["gate"], res_scale=x["c"],
                                     eps=1e-5)
    for a, b in zip(got, again):
        assert a is None and b is None or torch.equal(a, b)


def test_backward_equals_differences():
    """fp32, a direction at a time: the loss's curvature times the step squared (1e-3 of a unit direction) and
    rounding (1e-6 of the terms over the step) both stay below 2e-3 of the terms' size."""
    x = make("f32", 6, 64, 2, True, seed=1)
    names = ["x", "b", "wa", "wb", "gate", "c"]
    call = lambda a: gdn().gdn_block_norm_fwd(a[0], a[1], a[2], a[3], gate=a[4], res_scale=a[5])   # noqa: E731

    def loss(a):
        r, n = call(a)
        return float((r.double() * x["gr"].double()).sum() + (n.double() * x["gn"].double()).sum())

    args = [x[n] for n in names]
    grads = gdn().gdn_block_norm_bwd(*args[:4], x["gr"], x["gn"], gate=args[4], res_scale=args[5])
    gen = torch.Generator().manual_seed(2)
    for i, g in enumerate(grads):
        d = torch.randn(args[i].shape, generator=gen).cuda()
        h = 1e-2
        up, down = ([a + s * h * d if j == i else a for j, a in enumerate(args)] for s in (1, -1))
        num, ana = (loss(up) - loss(down)) / (2 * h), float((g.double() * d.double()).sum())
        size = float((g.double().abs() * d.double().abs()).sum())
        assert abs(num - ana) <= 2e-3 * size, (names[i], num, ana)


def test_in_place_strange_rows_and_streams():
    x = make("bf16", 9, 512, 2, True, seed=3)
    want = gdn().gdn_block_norm_fwd(x["x"], x["b"], x["wa"], x["wb"], gate=x["gate"], res_scale=x["c"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    xs, bs = x["x"].clone(), x["b"].clone()
    side.wait_stream(torch.cuda.current_stream())
    r, n = gdn().gdn_block_norm_fwd(xs, bs, x["wa"], x["wb"], gate=x["gate"], res_scale=x["c"], out=(xs, bs), stream=side)
    side.synchronize()
    assert r.data_ptr() == xs.data_ptr() and torch.equal(want[0], r) and torch.equal(want[1], n)
    # rows of zeros, a NaN, an infinite logit: they stay in their rows
    x["x"][2], x["b"][2], x["b"][4, 7] = 0, 0, float("nan")
    x["gate"][6], x["gate"][7] = float("inf"), -float("inf")
    r, n = gdn().gdn_block_norm_fwd(x["x"], x["b"], x["wa"], x["wb"], gate=x["gate"], res_scale=x["c"])
    keep = [i for i in range(9) if i != 4]
    rw, nw = od.block_norm(*(f64(x[m])[keep] for m in ("x", "b")), f64(x["wa"]), f64(x["wb"]), f64(x["gate"])[keep], f64(x["c"]))
    close(rw, r[keep], TOL["bf16"], "r")
    close(nw, n[keep], TOL["bf16"], "n")
    assert torch.isnan(r[4]).all() and torch.equal(r[7], x["x"][7])
    g = gdn().gdn_block_norm_bwd(x["x"], x["b"], x["wa"], x["wb"], x["gr"], x["gn"], gate=x["gate"], res_scale=x["c"])
    assert all(torch.isfinite(t[keep]).all() for t in (g[0], g[1], g[4]))


def test_no_rows_and_refusals():
    x = make("f32", 0, 64, 1, True)
    r, n = gdn().gdn_block_norm_fwd(x["x"], x["b"], x["wa"], x["wb"], gate=x["gate"], res_scale=x["c"])
    assert r.shape == (0, 64)
    gx, gb, ga, gw, gg, gc = gdn().gdn_block_norm_bwd(x["x"], x["b"], x["wa"], x["wb"], x["gr"], x["gn"], gate=x["gate"],
                                                      res_scale=x["c"])
    assert not ga.any() and not gw.any() and not gc.any() and gg.shape == (0, 1)
    x = make("f32", 4, 64, 1, True)
    f = gdn().gdn_block_norm_fwd
    for bad in (dict(b=x["b"][:, :32]), dict(b=x["b"].bfloat16()), dict(x=x["x"].t().contiguous().t()),
                dict(post_weight=x["wa"].bfloat16()), dict(pre_weight=x["wb"][:8]), dict(gate=x["x"][:, :2].contiguous()),
                dict(res_scale=x["c"].double()), dict(out=(x["x"], x["b"].bfloat16())), dict(b=x["b"].cpu())):
        a = dict(x=x["x"], b=x["b"], post_weight=x["wa"], pre_weight=x["wb"]) | bad
        with pytest.raises((ValueError, TypeError)):
            f(**a)
    for D in (12, 8200):
        y = make("f32", 1, D, 0, False)
        with pytest.raises(gdn().GdnError):
            f(y["x"], y["b"], y["wa"], y["wb"])
    with pytest.raises(gdn().GdnError):
        f(x["x"], x["b"], x["wa"], x["wb"], eps=-1.0)
