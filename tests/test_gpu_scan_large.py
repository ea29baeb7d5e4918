"""GPU: the selective scan where element offsets pass 2^31, and where many short or one very long sequence make more
segments than a block joins at once.  The far end is checked against the same tokens alone, from the state before them
(fp32 states good to the scan's own roundings, 2^-21 (4 + sqrt(T)) of the largest value for T tokens)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def gdn():
    import gated_deltanet_recurrence_03_gb300 as g
    return g


def make(T, D, N, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=dtype)   # noqa: E731
    f = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    return dict(u=n(1, T, D), delta=n(1, T, D), A_log=torch.log(torch.arange(1.0, N + 1, device="cuda")).expand(D, N) + 0.1 * f(D, N),
                B=n(1, T, 1, N), C=n(1, T, 1, N)), dict(skip=f(D), dt_bias=f(D) - 4, z=n(1, T, D))


def rel(a, b):
    return float((a.double() - b.double()).abs().max() / b.double().abs().max())


def test_offsets_past_32_bits():
    T, D, N, cut = 280_000, 8192, 8, 300   # 2.3e9 values a tensor
    x, parts = make(T, D, N, torch.bfloat16)
    assert T * D > 2 ** 31
    gy = torch.randn(1, T, D, device="cuda", dtype=torch.bfloat16, generator=torch.Generator(device="cuda").manual_seed(1))
    tail = lambda t: t[:, T - cut:].contiguous()   # noqa: E731
    xt = {k: (v if k == "A_log" else tail(v)) for k, v in x.items()}
    pt = {k: (tail(v) if k == "z" else v) for k, v in parts.items()}
    y, h = gdn().gdn_selective_scan_fwd(**x, **parts)
    head = lambda t: t[:, :T - cut]   # noqa: E731
    _, before = gdn().gdn_selective_scan_fwd(**{k: (v if k == "A_log" else head(v)) for k, v in x.items()},
                                             **{k: (head(v) if k == "z" else v) for k, v in parts.items()})
    yt, ht = gdn().gdn_selective_scan_fwd(**xt, h0=before, **pt)
    tol = 2.0 ** -21 * (4 + T ** 0.5)
    assert rel(h, ht) <= tol and rel(y[:, T - cut:], yt) <= 2.0 ** -8
    del y
    g = gdn().gdn_selective_scan_bwd(x["u"], x["delta"], x["A_log"], x["B"], x["C"], None, gy, None, want_grad_h0=False, **parts)
    gt = gdn().gdn_selective_scan_bwd(xt["u"], xt["delta"], xt["A_log"], xt["B"], xt["C"], before, tail(gy), None, **pt)
    for i in (0, 1, 3, 4, 7):   # u, delta, B, C, z: the last tokens' depend on nothing behind them
        assert rel(g[i][:, T - cut:], gt[i]) <= 2.0 ** -7, i


def test_many_segments_and_many_sequences():
    T, D, N = 200_000, 16, 16
    x, parts = make(T, D, N, torch.float32, seed=2)
    whole, h = gdn().gdn_selective_scan_fwd(**x, **parts)
    tol = 2.0 ** -21 * (4 + T ** 0.5)
    state, at = None, 0
    for n in (70_000, 129_000, 1000):
        cut = lambda t: t[:, at:at + n].contiguous()   # noqa: E731
        y, state = gdn().gdn_selective_scan_fwd(**{k: (v if k == "A_log" else cut(v)) for k, v in x.items()}, h0=state,
                                                **{k: (cut(v) if k == "z" else v) for k, v in parts.items()})
        assert rel(whole[:, at:at + n], y) <= tol
        at += n
    assert rel(h, state) <= tol
    # 20,000 sequences of 10 tokens are a batch of them
    cu = torch.arange(0, T + 1, 10, dtype=torch.int32, device="cuda")
    batch = lambda t: t.view(T // 10, 10, *t.shape[2:])   # noqa: E731
    gy = torch.randn(1, T, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    y, h = gdn().gdn_selective_scan_fwd(**x, cu_seqlens=cu, **parts)
    xb = {k: (v if k == "A_log" else batch(v)) for k, v in x.items()}
    pb = {k: (batch(v) if k == "z" else v) for k, v in parts.items()}
    yb, hb = gdn().gdn_selective_scan_fwd(**xb, **pb)
    assert rel(batch(y), yb) <= 1e-6 and rel(h, hb) <= 1e-6
    g = gdn().gdn_selective_scan_bwd(*x.values(), None, gy, h, cu_seqlens=cu, **parts)
    gb = gdn().gdn_selective_scan_bwd(*xb.values(), None, batch(gy), h, **pb)
    for i, (a, b) in enumerate(zip(g, gb)):
        assert rel(batch(a) if i in (0, 1, 3, 4, 7) else a, b) <= 2e-5, i
