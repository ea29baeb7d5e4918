"""GPU: the selective state space scan (prompt, token step, gradients) against oracle.scan's fp64 statement.

Tolerances are relative to the largest value of a channel (token results), of a state or of a tensor.  fp32 path: a
token's step multiplies by a decay good to 2^-22 and rounds twice, 2^-24 each, so T tokens leave at most 4 T 2^-24 of the
values that went in and, independent as these are, about 4 sqrt(T) 2^-24; sums over N states and the few functions of a
token add some 2^-22 more.  Held to 2^-21 (4 + sqrt(T)), four times that for gradients, whose sums run over two such
scans and over tokens or channels.  bf16 results: half a step of the result, 2^-9 of the value, held to 2^-8."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import scan as os_   # noqa: E402

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOKEN = ("u", "delta", "B", "C", "z")
NAMES = ("u", "delta", "A_log", "B", "C", "skip", "dt_bias", "z", "h0")


def gdn():
    import gated_deltanet_recurrence_03_gb300 as g
    return g


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make(dtype, lens, D, G, N, packed=False, gate=True, skip=True, bias=True, state=True, seed=0):
    """A layer's tensors: B and C slices of one projection, z the second half of the rows of another."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    B, T = (1, sum(lens)) if packed else (len(lens), lens[0])
    dt = DT[dtype]
    proj, xz = n(B, T, 16 + 2 * G * N).to(dt).cuda(), n(B, T, 2 * D).to(dt).cuda()
    step = torch.exp(np.log(1e-3) + np.log(100.0) * torch.rand(D, generator=gen))
    x = dict(u=n(B, T, D).to(dt).cuda(), delta=(0.5 * n(B, T, D)).to(dt).cuda(),
             A_log=(torch.log(torch.arange(1.0, N + 1)) + 0.1 * n(D, N)).cuda(),
             B=proj[..., 16:16 + G * N].unflatten(-1, (G, N)), C=proj[..., 16 + G * N:].unflatten(-1, (G, N)),
             skip=n(D).cuda() if skip else None,
             dt_bias=(step + torch.log(-torch.expm1(-step))).cuda() if bias else None, z=xz[..., D:] if gate else None,
             h0=n(len(lens), D, N).cuda() if state else None)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda() if packed else None
    return x, cu, n(B, T, D).to(dt).cuda(), n(len(lens), D, N).cuda() if state else None


def call(x, cu=None, **kw):
    return gdn().gdn_selective_scan_fwd(x["u"], x["delta"], x["A_log"], x["B"], x["C"], x["h0"], skip=x["skip"],
                                        dt_bias=x["dt_bias"], z=x["z"], cu_seqlens=cu, **kw)


def call_bwd(x, gy, gh, cu=None, **kw):
    return gdn().gdn_selective_scan_bwd(x["u"], x["delta"], x["A_log"], x["B"], x["C"], x["h0"], gy, gh, skip=x["skip"],
                                        dt_bias=x["dt_bias"], z=x["z"], cu_seqlens=cu, **kw)


def oracle_args(x):
    return {k: f64(v) for k, v in x.items()}


def close(want, got, tol, what, over=None):
    """Largest error over the largest value: of the tensor, or along the axes ``over`` where these have 64 values at
    least.  With fewer a channel's results may all be sums that cancel, while what bounds their rounding is their terms:
    the one d(delta) of a channel and token is u q + sum_n A w, found as 0.01154 from terms of about 1, each good to 2^-22."""
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if not want.size:
        return
    if over and np.prod([want.shape[i] for i in over]) < 64:
        over = None
    size = np.maximum(np.abs(want).max(over, keepdims=over is not None), 1e-30)
    err = (np.abs(got - want) / size).max()
    assert err <= tol, f"{what}: {err:.3e} > {tol:.1e}"


def tol32(T):
    return 2.0 ** -21 * (4 + T ** 0.5)


SHAPES = [   # lens, packed, D, G, N
    ((1,), False, 8, 1, 16), ((7, 7), False, 24, 1, 8), ((16,), False, 32, 1, 16), ((17, 17, 17), False, 72, 3, 32),
    ((8,), False, 40, 1, 64), ((128,), False, 64, 2, 16), ((129,), False, 136, 1, 16), ((300, 300), False, 48, 2, 8),
    ((700,), False, 520, 1, 16), ((260,), False, 16, 1, 64), ((5, 0, 129, 1, 64), True, 80, 2, 16),
    ((0, 0, 1), True, 16, 1, 8), ((256, 128, 1, 0, 257), True, 32, 1, 32), ((640, 3, 513), True, 56, 1, 16),
    ((130, 2), True, 112, 7, 64), ((33,), False, 4864, 1, 16), ((0, 0), False, 16, 1, 16),
]
CASES = [(dtype, *s, opt) for i, s in enumerate(SHAPES) for dtype, opt in
         (("f32", i % 4), ("bf16", (i + 1) % 4))]
OPTIONS = [dict(), dict(gate=False), dict(skip=False, bias=False), dict(gate=False, skip=False, state=False)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(case):
    dtype, lens, packed, D, G, N, opt = case
    x, cu, gy, gh = make(dtype, lens, D, G, N, packed, **OPTIONS[opt])
    t32, small = tol32(max(lens)), 2.0 ** -8 if dtype == "bf16" else None
    y, hf = call(x, cu)
    want_y, want_h = os_.forward(**oracle_args(x), cu=None if cu is None else cu.tolist())
    close(want_y, y, small or t32, "y", (0, 1))
    close(want_h, hf, t32, "h_final", (2,))
    got = call_bwd(x, gy, gh, cu)
    a = oracle_args(x)
    want = os_.backward(a["u"], a["delta"], a["A_log"], a["B"], a["C"], f64(gy), a["h0"], f64(gh), a["skip"], a["dt_bias"],
                        a["z"], None if cu is None else cu.tolist())
    for name, w, g in zip(NAMES, want, got):
        if name in ("skip", "dt_bias", "z") and x[name] is None:
            assert g is None, name
        elif name in TOKEN:
            assert g.dtype == DT[dtype]
            close(w, g, small or 4 * t32, "grad_" + name, (0, 1))
        else:
            close(w, g, 4 * t32, "grad_" + name)
    for a, b in zip((y, hf, *got), (*call(x, cu), *call_bwd(x, gy, gh, cu))):
        assert (a is None and b is None) or torch.equal(a, b)


def test_long_rows_in_segments_and_whole():
    """A sequence that one block walks, and the same among others in segments."""
    x, _, gy, gh = make("f32", (2100,), 24, 1, 16)
    y, hf = call(x)
    want_y, want_h = os_.forward(**oracle_args(x))
    close(want_y, y, tol32(2100), "y", (0, 1))
    close(want_h, hf, tol32(2100), "h", (2,))
    wide = {k: v for k, v in x.items()}
    rep = 224   # 24 x 224 channels: no segments
    for k in ("u", "delta", "z"):
        wide[k] = x[k].repeat(1, 1, rep)
    for k in ("A_log", "skip", "dt_bias"):
        wide[k] = x[k].repeat(rep, *[1] * (x[k].dim() - 1))
    wide["h0"] = x["h0"].repeat(1, rep, 1)
    y2, h2 = call(wide)
    assert torch.equal(y2[..., :24], y2[..., -24:])
    close(want_y, y2[..., 24:48], tol32(2100), "y", (0, 1))
    close(want_h, h2[:, :24], tol32(2100), "h", (2,))


def test_backward_equals_differences():
    """fp32, a direction at a time: the loss's curvature times the step squared and rounding over the step both stay
    below 2e-3 of the terms' size (the step is 1e-2 of a unit direction)."""
    x, cu, gy, gh = make("f32", (40, 0, 90), 16, 2, 8, packed=True, seed=1)
    grads = call_bwd(x, gy, gh, cu)
    gen = torch.Generator().manual_seed(2)

    def loss(v):
        y, h = call(v, cu)
        return float((y.double() * gy.double()).sum() + (h.double() * gh.double()).sum())

    for name, g in zip(NAMES, grads):
        d = torch.randn(x[name].shape, generator=gen).cuda()
        h = 1e-2
        up, down = ({**x, name: x[name] + s * h * d} for s in (1, -1))
        num, ana = (loss(up) - loss(down)) / (2 * h), float((g.double() * d.double()).sum())
        size = float((g.double().abs() * d.double().abs()).sum())
        assert abs(num - ana) <= 2e-3 * size, (name, num, ana)


def test_given_results_slices_and_in_place_states():
    x, cu, gy, gh = make("bf16", (100, 0, 57), 48, 2, 16, packed=True)
    y, hf = call(x, cu)
    out, keep = torch.empty_like(y), x["h0"].clone()
    y2, h2 = call({**x, "h0": keep}, cu, out=out, h_final=keep)
    assert y2 is out and torch.equal(y, y2) and h2 is keep and torch.equal(hf, keep)
    assert call(x, cu, output_final_state=False)[1] is None
    want = call_bwd(x, gy, gh, cu)
    T = x["u"].shape[1]
    proj, xz = torch.full((1, T, 96), 7.0).bfloat16().cuda(), torch.full((1, T, 96), 7.0).bfloat16().cuda()
    views = (proj[..., 16:48].unflatten(-1, (2, 16)), proj[..., 64:].unflatten(-1, (2, 16)), xz[..., 48:])
    got = call_bwd(x, gy, gh, cu, grads=views)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert (proj[..., :16] == 7).all() and (proj[..., 48:64] == 7).all() and (xz[..., :48] == 7).all()
    assert call_bwd(x, gy, gh, cu, want_grad_h0=False)[8] is None
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    assert torch.equal(call(x, cu, workspace=ws)[0], y)
    for a, b in zip(want, call_bwd(x, gy, gh, cu, workspace=ws)):
        assert torch.equal(a, b)


def test_rows_of_no_sequence_are_left_alone():
    x, _, gy, gh = make("f32", (60, 40, 200), 24, 1, 8, packed=True)
    cu = torch.tensor([0, 60, 100, 270], dtype=torch.int32).cuda()   # 30 rows behind the last sequence
    y = torch.full_like(x["u"], 7.0)
    call(x, cu, out=y)
    want, _ = os_.forward(**oracle_args(x), cu=cu.tolist())
    close(want[:, :270], y[:, :270], tol32(200), "y", (0, 1))
    assert (y[:, 270:] == 7).all()
    gB, gC, gz = (torch.full_like(x[n].contiguous(), 7.0) for n in ("B", "C", "z"))
    got = call_bwd(x, gy, gh, cu, grads=(gB, gC, gz))
    a = oracle_args(x)
    ref = os_.backward(a["u"], a["delta"], a["A_log"], a["B"], a["C"], f64(gy), a["h0"], f64(gh), a["skip"], a["dt_bias"],
                       a["z"], cu.tolist())
    assert all((t[:, 270:] == 7).all() for t in (gB, gC, gz))
    close(ref[2], got[2], 4 * tol32(200), "A_log")
    close(ref[3][:, :270], gB[:, :270], 4 * tol32(200), "B", (0, 1))
    # the weights' sums take the rows of the sequences alone
    z = a["z"][:, :270]
    p = f64(gy)[:, :270] * z / (1 + np.exp(-z))
    close((p * a["u"][:, :270]).sum((0, 1)), got[5], 4 * tol32(200), "skip")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D,G,N", [(1, 8, 1, 16), (3, 72, 3, 8), (37, 136, 1, 16), (5, 48, 2, 32), (2, 40, 1, 64),
                                        (300, 1032, 1, 16)])
def test_step(dtype, rows, D, G, N):
    # the exponent x = dt A is off by x 2^-20.5 at most (dt and A by 2^-22 each and the rounding of their product), the
    # decay so by x e^-x 2^-20.5 <= 2^-21.9, and with the roundings of h each term C h by 2^-21 of itself.  A result is
    # the sum of N such terms, whose sizes add up to some 4 times the largest result of the row, 8 with 64 states: 2^-18.
    t32 = 2.0 ** -18
    x, _, _, _ = make(dtype, (rows,), D, G, N, seed=3)
    row = {k: (v[0] if k in TOKEN else v) for k, v in x.items() if k != "h0"}
    pool = torch.randn(rows + 9, D, N, generator=torch.Generator().manual_seed(4)).cuda()
    slots = torch.randperm(rows + 9, generator=torch.Generator().manual_seed(5))[:rows].to(torch.int32).cuda()
    if rows > 2:
        slots[1], slots[-1] = -1, rows + 9
    h = pool.clone()
    args = (row["u"], row["delta"], row["A_log"], row["B"], row["C"])
    parts = dict(skip=row["skip"], dt_bias=row["dt_bias"], z=row["z"])
    y = gdn().gdn_selective_scan_step(*args, h, slots=slots, **parts)
    want_y, want_h = os_.step(**{k: f64(v) for k, v in row.items()}, h=f64(pool), slots=slots.tolist())
    close(want_y, y, 2.0 ** -8 if dtype == "bf16" else t32, "y", (1,))
    close(want_h, h, t32, "h", (2,))
    idle = [i for i in range(rows + 9) if i not in slots.tolist()]
    assert torch.equal(h[idle], pool[idle])
    if rows > 2:
        assert not y[1].any() and not y[-1].any()
    h2 = pool[:rows].clone()
    y2 = gdn().gdn_selective_scan_step(*args, h2, out=torch.empty_like(y), **parts)
    want_y, want_h = os_.step(**{k: f64(v) for k, v in row.items()}, h=f64(pool[:rows]))
    close(want_y, y2, 2.0 ** -8 if dtype == "bf16" else t32, "y", (1,))
    close(want_h, h2, t32, "h", (2,))
    # without the parts
    h3 = pool[:rows].clone()
    y3 = gdn().gdn_selective_scan_step(*args, h3)
    bare = {k: f64(row[k]) for k in ("u", "delta", "A_log", "B", "C")}
    close(os_.step(**bare, h=f64(pool[:rows]))[0], y3, 2.0 ** -8 if dtype == "bf16" else t32, "y", (1,))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_then_tokens(dtype):
    x, _, _, _ = make(dtype, (45, 45), 72, 1, 16, seed=6)
    whole, last = call(x)
    cut = lambda s: {k: (v[:, s] if k in TOKEN else v) for k, v in x.items()}   # noqa: E731
    first = cut(slice(0, 40))
    first["u"], first["delta"] = first["u"].contiguous(), first["delta"].contiguous()
    for k in ("B", "C", "z"):
        first[k] = first[k].contiguous()
    y, h = call(first)
    close(f64(whole[:, :40]), y, 2.0 ** -8 if dtype == "bf16" else 1e-6, "prompt", (0, 1))
    for t in range(40, 45):
        r = cut(t)
        y = gdn().gdn_selective_scan_step(r["u"], r["delta"], r["A_log"], r["B"], r["C"], h, skip=r["skip"],
                                          dt_bias=r["dt_bias"], z=r["z"])
        close(f64(whole[:, t]), y, 2.0 ** -7 if dtype == "bf16" else 1e-5, f"token {t}")
    close(f64(last), h, tol32(45), "state", (2,))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["u", "delta", "z"])
def test_what_is_not_finite_stays_in_its_channel(value, what):
    """A token of one channel: other channels, other sequences and earlier outputs of its own keep every bit."""
    x, cu, gy, gh = make("f32", (300, 300, 5), 40, 1, 16, packed=True, seed=7)
    base, base_g = call(x, cu), call_bwd(x, gy, gh, cu)
    bad = {**x, what: x[what].clone()}
    bad[what][0, 450, 11] = value
    got, got_g = call(bad, cu), call_bwd(bad, gy, gh, cu)
    others = [c for c in range(40) if c != 11]
    assert torch.equal(base[0][..., others], got[0][..., others]) and torch.equal(base[1][:, others], got[1][:, others])
    assert torch.equal(base[0][:, :450, 11], got[0][:, :450, 11]) and torch.equal(base[0][:, 600:], got[0][:, 600:])
    assert torch.equal(base[1][[0, 2]], got[1][[0, 2]])
    for name, a, b in zip(NAMES, base_g, got_g):
        if name in ("u", "delta", "z"):
            assert torch.equal(a[..., others], b[..., others]), name
            assert torch.equal(a[:, :300], b[:, :300]) and torch.equal(a[:, 600:], b[:, 600:]), name
        elif name in ("A_log", "skip", "dt_bias"):
            assert torch.equal(a[others], b[others]), name
        elif name in ("B", "C"):
            assert torch.equal(a[:, :300], b[:, :300]) and torch.equal(a[:, 600:], b[:, 600:]), name
    y = os_.forward(**oracle_args(bad), cu=cu.tolist())[0]
    with np.errstate(all="ignore"):
        assert np.array_equal(np.isfinite(y), np.isfinite(f64(got[0])))


def test_rates_of_any_size():
    """A_log of +-inf and beyond fp32's exponentials: no decay, or nothing kept; ragged ends stay clean."""
    x, cu, gy, gh = make("f32", (21, 300), 16, 1, 8, packed=True, seed=8)
    x["A_log"][3], x["A_log"][5], x["A_log"][7] = -float("inf"), 200.0, 88.5
    y, h = call(x, cu)
    a = oracle_args(x)
    a["A_log"][5] = 60.0   # the decays are zero either way
    a["A_log"][7] = 60.0
    want_y, want_h = os_.forward(**a, cu=cu.tolist())
    close(want_y, y, tol32(300), "y", (0, 1))
    close(want_h, h, tol32(300), "h", (2,))
    assert all(torch.isfinite(g).all() for n, g in zip(NAMES, call_bwd(x, gy, gh, cu)) if n != "A_log")


def test_large_steps_and_small_ones():
    """softplus far on both sides: dt from 1e-13 to 60."""
    x, _, _, _ = make("f32", (64,), 16, 1, 8, bias=False, seed=9)
    x["delta"] = torch.linspace(-30, 60, 64 * 16).view(1, 64, 16).cuda()
    y, h = call(x)
    want_y, want_h = os_.forward(**oracle_args(x))
    close(want_y, y, tol32(64), "y", (0, 1))
    close(want_h, h, tol32(64), "h", (2,))


def calls():
    x, cu, gy, gh = make("bf16", (700, 3), 64, 1, 16, packed=True, seed=10)
    row = {k: (v[0, :5] if k in TOKEN else v) for k, v in x.items()}
    pool = torch.randn(5, 64, 16, generator=torch.Generator().manual_seed(11)).cuda()

    def step(**o):
        h = pool.clone()
        if "stream" in o:
            o["stream"].wait_stream(torch.cuda.current_stream())
        return gdn().gdn_selective_scan_step(row["u"], row["delta"], row["A_log"], row["B"], row["C"], h, skip=row["skip"],
                                             dt_bias=row["dt_bias"], z=row["z"], **o), h
    return {"fwd": lambda **o: call(x, cu, **o), "bwd": lambda **o: call_bwd(x, gy, gh, cu, **o), "step": step}


@pytest.mark.parametrize("name", ["fwd", "bwd", "step"])
def test_in_a_graph_and_on_another_stream(name):
    f = calls()[name]
    want = [t.clone() for t in f()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = f(stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["fwd", "bwd"])
def test_new_tensors_are_not_in_use_on_another_stream(name):
    f = calls()[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in f()]
    f(stream=side)   # its memory is in the allocator's pools from here on
    torch.cuda.synchronize()
    blocks = [torch.empty_like(t) for t in want for _ in range(4)]
    torch.cuda._sleep(100_000_000)   # tens of milliseconds before the writes below
    for t in blocks:
        t.fill_(7.0)
    del blocks, t
    got = f(stream=side)
    torch.cuda.synchronize()
    for w, r in zip(want, got):
        assert torch.equal(w, r), name


def test_refusals():
    x, cu, gy, gh = make("f32", (20,), 16, 1, 8)
    bad = [dict(delta=x["delta"][:, :10]), dict(delta=x["delta"].bfloat16()), dict(u=x["u"].double()), dict(B=x["B"][..., :4]),
           dict(C=x["C"].bfloat16()), dict(A_log=x["A_log"].bfloat16()), dict(A_log=x["A_log"][:8]), dict(skip=x["skip"][:8]),
           dict(z=x["z"].cpu()), dict(h0=x["h0"][:, :8]), dict(u=x["u"].expand(1, 20, 16)[:, :, ::2])]
    for b in bad:
        with pytest.raises((ValueError, TypeError)):
            call({**x, **b})
    with pytest.raises((ValueError, TypeError)):
        call_bwd(x, gy.bfloat16(), gh)
    with pytest.raises(ValueError):
        call_bwd(x, gy, gh, grads=(x["B"].contiguous(), x["C"].contiguous(), None))
    y, _, _, _ = make("f32", (20,), 16, 1, 8)
    y["A_log"], y["B"], y["C"], y["h0"] = (torch.zeros(*s, device="cuda") for s in
                                           ((16, 12), (1, 20, 1, 12), (1, 20, 1, 12), (1, 16, 12)))
    with pytest.raises(gdn().GdnError, match="not in"):
        call(y)
    z, _, _, _ = make("f32", (20,), 12, 1, 8)
    with pytest.raises(gdn().GdnError, match="multiple of 8"):
        call(z)
