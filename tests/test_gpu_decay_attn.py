"""GPU: linear attention with a decay for each value head (prompt form, token step, backward) against the
fp64 token loop of oracle.decay.

Tolerances (max error over max value).  fp32: every sum is fp32 with products exact to 2^-22 or better;
a sum of n terms is off by about sqrt(n) 2^-24 of its size, n the head's memory (at most about 2000 tokens x
128 features): 1e-5.  bf16 results: the rounding of the result and of two operands of the tensor cores (the
masked scores and the state), each at most 2^-8 of a term and averaging out over a row: 2^-7, 8e-3.  States of
bf16 inputs are sums in fp32 accuracy: 1e-5."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import decay as od   # noqa: E402

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 1e-5, "bf16": 8e-3}
STATE_TOL = 1e-5


def gdn():
    import gated_deltanet_recurrence_03_gb300 as g
    return g


def close(want, got, tol, what=""):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if want.size:
        err = np.abs(got - want).max() / max(np.abs(want).max(), 1e-30)
        assert err <= tol, f"{what}: {err:.3e} > {tol:.1e}"   # a NaN fails too


def f64(t):
    return t.double().cpu().numpy()


def make(dtype, lens, packed, Hqk, Hv, dk, dv, seed=0, strided=False, slope=(1.0, 9.0)):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    B, T = (1, sum(lens)) if packed else (len(lens), lens[0])
    if strided:   # slices of one packed projection, with channels that are none of q, k, v behind them
        p = n(B, T, 2 * Hqk * dk + Hv * dv + 32).to(DT[dtype]).cuda()
        q, k, v, _ = p.split([Hqk * dk, Hqk * dk, Hv * dv, 32], -1)
        q, k, v = q.unflatten(-1, (Hqk, dk)), k.unflatten(-1, (Hqk, dk)), v.unflatten(-1, (Hv, dv))
    else:
        q, k, v = (n(B, T, h, d).to(DT[dtype]).cuda() for h, d in ((Hqk, dk), (Hqk, dk), (Hv, dv)))
    ns = len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32) if packed else None
    return dict(q=q, k=k, v=v, g=-torch.exp2(-torch.linspace(*slope, Hv)).cuda(), S0=(4 * n(ns, Hv, dk, dv)).cuda(),
                do=n(B, T, Hv, dv).to(DT[dtype]).cuda(), dS=n(ns, Hv, dk, dv).cuda(), cu=cu,
                cu_dev=None if cu is None else torch.from_numpy(cu).cuda(), scale=dk ** -0.5)


SHAPES = [   # dtype, lens, packed, Hqk, Hv, dk, dv, strided
    ("bf16", [1], False, 1, 1, 128, 128, False),
    ("bf16", [77], False, 2, 4, 128, 128, True),
    ("bf16", [128, 128], False, 1, 1, 128, 128, False),
    ("bf16", [129, 0, 1, 300, 64, 63], True, 2, 6, 128, 128, True),
    ("bf16", [700], False, 1, 2, 128, 128, False),
    ("bf16", [0, 0, 257], True, 1, 1, 128, 128, False),
    ("bf16", [200, 65], True, 2, 2, 64, 64, True),
    ("bf16", [131] * 3, False, 3, 3, 32, 32, False),
    ("bf16", [90, 1], True, 1, 2, 64, 128, False),
    ("f32", [1, 0, 2], True, 1, 2, 32, 64, True),
    ("f32", [515], False, 2, 4, 64, 64, True),
    ("f32", [64, 65, 63], True, 1, 1, 128, 128, False),
    ("f32", [140, 140], False, 1, 3, 128, 32, False),
]
IDS = ["-".join([s[0], "x".join(map(str, s[1])), f"h{s[3]}:{s[4]}", f"d{s[5]}:{s[6]}"]) for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("state", [False, True])
def test_forward(shape, state):
    dtype, strided = shape[0], shape[-1]
    x = make(*shape[:-1], strided=strided)
    S0 = x["S0"] if state else None
    out, S = gdn().gdn_decay_attn_fwd(x["q"], x["k"], x["v"], x["g"], S0, scale=x["scale"], cu_seqlens=x["cu_dev"])
    gdn().check_device_status()
    want, Sw = od.forward(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["g"]), f64(S0) if state else None, x["scale"],
                          x["cu"])
    assert out.dtype == DT[dtype] and S.dtype == torch.float32
    close(want, out, TOL[dtype], "out")
    close(Sw, S, STATE_TOL, "S_final")


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("state", [False, True])
def test_backward(shape, state):
    dtype, strided = shape[0], shape[-1]
    x = make(*shape[:-1], seed=1, strided=strided)
    S0, dS = (x["S0"], x["dS"]) if state else (None, None)
    got = gdn().gdn_decay_attn_bwd(x["q"], x["k"], x["v"], x["g"], S0, x["do"], dS, scale=x["scale"],
                                   cu_seqlens=x["cu_dev"])
    gdn().check_device_status()
    want = od.backward(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["g"]), f64(x["do"]), f64(S0) if state else None,
                       f64(dS) if state else None, x["scale"], x["cu"])
    for name, w, g in zip(("grad_q", "grad_k", "grad_v"), want, got):
        assert g.dtype == DT[dtype]
        close(w, g, TOL[dtype], name)
    close(want[3], got[3], STATE_TOL, "grad_S0")


def test_backward_equals_differences_of_the_forward():
    """fp32: the gradient's product with a direction against the central difference of the loss along it.
    The loss is linear in v and S0 and, for one of q, k at a time, linear too: any step size is exact but
    for rounding, about 1e-6 of the sum's terms."""
    x = make("f32", [70, 0, 33], True, 1, 2, 64, 32, seed=2)
    gen = torch.Generator().manual_seed(3)

    def loss(q, k, v, S0):
        o, S = gdn().gdn_decay_attn_fwd(q, k, v, x["g"], S0, scale=0.3, cu_seqlens=x["cu_dev"])
        return float((o.double() * x["do"].double()).sum() + (S.double() * x["dS"].double()).sum())

    args = [x["q"], x["k"], x["v"], x["S0"]]
    grads = gdn().gdn_decay_attn_bwd(*args[:3], x["g"], x["S0"], x["do"], x["dS"], scale=0.3, cu_seqlens=x["cu_dev"])
    for i, g in enumerate(grads):
        d = torch.randn(args[i].shape, generator=gen).cuda()
        up, down = ([a + s * d if j == i else a for j, a in enumerate(args)] for s in (1.0, -1.0))
        num, ana = (loss(*up) - loss(*down)) / 2, float((g.double() * d.double()).sum())
        size = float((g.double().abs() * d.double().abs()).sum())
        assert abs(num - ana) <= 1e-4 * size, (i, num, ana)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 32), ("f32", 64)])
def test_decays_from_none_to_all(dtype, d):
    """A head that never forgets (0), ones that forget at once (-inf, -1000) and strong ones between."""
    x = make(dtype, [200], False, 1, 6, d, d, seed=4)
    x["g"] = torch.tensor([0.0, -float("inf"), -1000.0, -30.0, -3.0, -1e-4]).cuda()
    out, S = gdn().gdn_decay_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], scale=x["scale"])
    want, Sw = od.forward(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["g"]), f64(x["S0"]), x["scale"])
    grads = gdn().gdn_decay_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["do"], x["dS"], scale=x["scale"])
    gw = od.backward(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["g"]), f64(x["do"]), f64(x["S0"]), f64(x["dS"]),
                     x["scale"])
    for h in range(6):
        close(want[:, :, h], out[:, :, h], TOL[dtype], f"out of head {h}")
        close(Sw[:, h], S[:, h], STATE_TOL, f"S_final of head {h}")
        close(gw[2][:, :, h], grads[2][:, :, h], TOL[dtype], f"grad_v of head {h}")
        close(gw[3][:, h], grads[3][:, h], STATE_TOL, f"grad_S0 of head {h}")
    close(gw[0], grads[0], TOL[dtype], "grad_q")
    close(gw[1], grads[1], TOL[dtype], "grad_k")


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 32)])
def test_a_sequence_with_nan_and_inf_leaves_the_others_alone(dtype, d):
    lens = [50, 70, 130, 9]
    x = make(dtype, lens, True, 1, 2, d, d, seed=5)
    run = lambda: (*gdn().gdn_decay_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], cu_seqlens=x["cu_dev"]),   # noqa: E731
                   *gdn().gdn_decay_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["do"], x["dS"],
                                             cu_seqlens=x["cu_dev"]))
    clean = run()
    bad = slice(50, 120)
    for n, value in (("q", float("inf")), ("k", float("nan")), ("v", float("nan")), ("do", -float("inf"))):
        x[n][0, bad] = value
    dirty = run()
    others = torch.tensor([0, 2, 3]).cuda()
    keep = torch.ones(sum(lens), dtype=torch.bool).cuda()
    keep[bad] = False
    for i, (a, b) in enumerate(zip(clean, dirty)):
        state = i in (1, 5)
        a, b = (a[others], b[others]) if state else (a[0, keep], b[0, keep])
        assert torch.equal(a, b), f"output {i}"


def test_no_tokens_and_no_sequences():
    for T, B in ((0, 2), (5, 0)):
        q, v = torch.zeros(B, T, 1, 32).cuda(), torch.zeros(B, T, 2, 64).cuda()
        g, S0 = -torch.ones(2).cuda(), torch.randn(B, 2, 32, 64).cuda()
        out, S = gdn().gdn_decay_attn_fwd(q, q, v, g, S0)
        assert out.shape == v.shape and torch.equal(S, S0)
        assert not gdn().gdn_decay_attn_fwd(q, q, v, g)[1].any()
        *_, dS0 = gdn().gdn_decay_attn_bwd(q, q, v, g, S0, v, S0)
        assert torch.equal(dS0, S0)
        assert gdn().gdn_decay_attn_bwd(q, q, v, g, None, v, None, want_grad_S0=False)[3] is None


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_state_in_place_resume_and_steps(dtype, d):
    """A prompt in two halves, the state handed over in place, then tokens one by one: the whole prompt."""
    x = make(dtype, [333], False, 2, 4, d, d, seed=6)
    whole, S = gdn().gdn_decay_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"])
    state = x["S0"].clone()
    part = lambda a, b: [x[n][:, a:b] for n in "qkv"]   # noqa: E731
    first, s1 = gdn().gdn_decay_attn_fwd(*part(0, 200), x["g"], state, S_final=state)
    second, _ = gdn().gdn_decay_attn_fwd(*part(200, 330), x["g"], state, S_final=state)
    assert s1.data_ptr() == state.data_ptr()
    last = [gdn().gdn_decay_attn_step(*(x[n][:, t] for n in "qkv"), x["g"], state) for t in range(330, 333)]
    got = torch.cat([first, second, torch.stack(last, 1)], 1)
    close(f64(whole), got, 2 * TOL[dtype], "outputs")
    close(f64(S), state, 2 * STATE_TOL, "state")


def test_outputs_given_strided_gradients_and_determinism():
    x = make("bf16", [150, 41], True, 2, 4, 128, 128, seed=7, strided=True)
    call = lambda **kw: gdn().gdn_decay_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["do"], x["dS"],   # noqa: E731
                                                 cu_seqlens=x["cu_dev"], **kw)
    a, b = call(), call()
    packed = torch.full((1, 191, 2 * 2 * 128 + 4 * 128), 7.0, dtype=torch.bfloat16).cuda()
    views = [t.unflatten(-1, (h, 128)) for t, h in zip(packed.split([256, 256, 512], -1), (2, 2, 4))]
    c = call(grads=views)
    for u, w, z in zip(a, b, c):
        assert torch.equal(u, w) and torch.equal(u, z)
    out = torch.empty_like(x["v"], memory_format=torch.contiguous_format)
    S = torch.empty_like(x["S0"])
    o1, S1 = gdn().gdn_decay_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], cu_seqlens=x["cu_dev"])
    o2, S2 = gdn().gdn_decay_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], cu_seqlens=x["cu_dev"], out=out, S_final=S)
    assert o2.data_ptr() == out.data_ptr() and torch.equal(o1, o2) and torch.equal(S1, S2)
    o3, none = gdn().gdn_decay_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], cu_seqlens=x["cu_dev"],
                                        output_final_state=False)
    assert none is None
    close(f64(o1), o3, TOL["bf16"], "out without the final state")


def test_on_another_stream():
    x = make("bf16", [300], False, 1, 2, 128, 128, seed=8)
    here, S = gdn().gdn_decay_attn_fwd(x["q"], x["k"], x["v"], x["g"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there, S2 = gdn().gdn_decay_attn_fwd(x["q"], x["k"], x["v"], x["g"], stream=side)
    side.synchronize()
    assert torch.equal(here, there) and torch.equal(S, S2)


def test_a_long_sequence_of_few_heads():
    """Many chunks one after another, split over the card: the state at the end and sampled outputs."""
    T, Hv, d = 20011, 2, 128
    x = make("bf16", [T, 1, 500], True, 1, Hv, d, d, seed=9, slope=(8.0, 12.0))
    out, S = gdn().gdn_decay_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], scale=x["scale"], cu_seqlens=x["cu_dev"])
    grads = gdn().gdn_decay_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["do"], x["dS"], scale=x["scale"],
                                     cu_seqlens=x["cu_dev"])
    args = [f64(x[n]) for n in ("q", "k", "v", "g")]
    want, Sw = od.forward(*args, f64(x["S0"]), x["scale"], x["cu"])
    close(want, out, TOL["bf16"], "out")
    close(Sw, S, STATE_TOL, "S_final")
    gw = od.backward(*args, f64(x["do"]), f64(x["S0"]), f64(x["dS"]), x["scale"], x["cu"])
    for name, w, g in zip(("grad_q", "grad_k", "grad_v"), gw, grads):
        close(w, g, TOL["bf16"], name)
    close(gw[3], grads[3], STATE_TOL, "grad_S0")


@pytest.mark.parametrize("dtype,N,Hqk,Hv,dk,dv", [("bf16", 1, 1, 1, 128, 128), ("bf16", 5, 2, 6, 128, 128),
                                                  ("bf16", 3, 1, 2, 64, 32), ("f32", 7, 2, 4, 32, 128),
                                                  ("f32", 2, 1, 1, 64, 64), ("f32", 130, 4, 8, 128, 64)])
@pytest.mark.parametrize("pooled", [False, True])
def test_step(dtype, N, Hqk, Hv, dk, dv, pooled):
    x = make(dtype, [1] * N, False, Hqk, Hv, dk, dv, seed=10, strided=True)
    q, k, v = (x[n][:, 0] for n in "qkv")
    S, slots = x["S0"], None
    if pooled:
        S = torch.randn(N + 9, Hv, dk, dv, generator=torch.Generator().manual_seed(1)).cuda()
        slots = torch.randperm(N + 9, generator=torch.Generator().manual_seed(2))[:N].to(torch.int32)
        slots[::3] = torch.tensor([-1, N + 9, -2 ** 31])[torch.arange(len(slots[::3])) % 3].to(torch.int32)
    want, Sw = od.step(f64(q), f64(k), f64(v), f64(x["g"]), f64(S), None if slots is None else slots.tolist(), 0.25)
    before = S.clone()
    out = gdn().gdn_decay_attn_step(q, k, v, x["g"], S, slots=None if slots is None else slots.cuda(), scale=0.25)
    close(want, out, TOL[dtype] if dtype == "f32" else 2.0 ** -8, "out")
    close(Sw, S, 1e-6, "S")
    if pooled:
        idle = [n for n, s in enumerate(slots.tolist()) if not 0 <= s < N + 9]
        assert not out[idle].any()
        untouched = sorted(set(range(N + 9)) - set(slots.tolist()))
        assert torch.equal(S[untouched], before[untouched])


def test_step_with_strong_decays_and_nan_in_an_idle_row():
    x = make("f32", [1] * 3, False, 1, 2, 64, 64, seed=11)
    x["g"] = torch.tensor([-float("inf"), 0.0]).cuda()
    q, k, v = (x[n][:, 0] for n in "qkv")
    k[1] = float("nan")
    S = x["S0"].clone()
    out = gdn().gdn_decay_attn_step(q, k, v, x["g"], S, slots=torch.tensor([2, -1, 0], dtype=torch.int32).cuda())
    want, Sw = od.step(f64(q), f64(k), f64(v), f64(x["g"]), f64(x["S0"]), [2, -1, 0])
    close(want, out, 1e-5, "out")
    close(Sw, S, 1e-6, "S")


def test_refusals_of_the_binding():
    x = make("bf16", [8], False, 1, 2, 64, 64)
    fwd, step, bwd = gdn().gdn_decay_attn_fwd, gdn().gdn_decay_attn_step, gdn().gdn_decay_attn_bwd
    q, k, v, g, S = x["q"], x["k"], x["v"], x["g"], x["S0"]
    for bad in (dict(q=q[0]), dict(k=k[:, :4]), dict(v=v.float()), dict(g=g.double()), dict(g=g[:1]), dict(S0=S[:, :1]),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2).expand(2, -1, -1, -1)),
                dict(v=v.flip(3).transpose(2, 3).contiguous().transpose(2, 3)), dict(q=q.half(), k=k.half(), v=v.half()),
                dict(cu_seqlens=torch.tensor([0, 8]).cuda()), dict(out=torch.empty(1, 8, 2, 64).cuda()),
                dict(v=v.cpu())):
        a = dict(q=q, k=k, v=v, g=g, S0=None) | bad
        with pytest.raises((ValueError, TypeError)):
            fwd(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("g"), a.pop("S0"), **a)
    with pytest.raises(gdn().GdnError):   # head dims the library does not take
        fwd(q[..., :48].contiguous(), k[..., :48].contiguous(), v, g)
    with pytest.raises(gdn().GdnError):   # three value heads over two query/key heads
        fwd(q.repeat(1, 1, 2, 1), k.repeat(1, 1, 2, 1), torch.cat([v, v[:, :, :1]], 2), torch.cat([g, g[:1]]))
    with pytest.raises(ValueError):
        step(q[:, 0], k[:, 0], v[:, 0], g, S[:, :, :32])
    with pytest.raises(ValueError):
        step(q[:, 0], k[:, 0], v[:, 0], g, S, slots=torch.zeros(1, dtype=torch.int64).cuda())
    with pytest.raises(ValueError):
        bwd(q, k, v, g, S, x["do"].float(), None)
    with pytest.raises(ValueError):
        bwd(q, k, v, g, S, x["do"], None, grads=(q, k, v[:, :4]))
