"""GPU: the decayed attention's and the block norm's forms that only larger calls take, each against fp64: fp32 scans of
64 columns a block, whole-state token steps, segments of every head dim, rings of one stage over many rows; and each
call captured in a CUDA graph and replayed on other inputs.  Tolerances as in test_gpu_decay_attn.py and
test_gpu_block_norm.py (the sums are of the same lengths)."""
import pytest

torch = pytest.importorskip("torch")

import test_gpu_block_norm as bn   # noqa: E402
from oracle import decay as od   # noqa: E402
from test_gpu_decay_attn import STATE_TOL, TOL, close, f64, gdn, make   # noqa: E402

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

PACKED, BATCH, LONG = [700, 0, 129, 1, 514], [70] * 20, [1500, 0, 37]
SCANS = (
    # at least 76 blocks of 64 columns: segments of a packed call, whole sequences of a batch
    [("f32", PACKED, True, 4, 8, dk, dv) for dk in (32, 64, 128) for dv in (64, 128)] +
    [("f32", BATCH, False, 4, 8, 64, 64), ("f32", BATCH, False, 8, 8, 128, 128)] +
    # segments: every head dim, and dk != dv, where the gradients take two launches over one workspace
    [("bf16", LONG, True, 1, 2, dk, dv) for dk, dv in ((32, 32), (64, 64), (128, 64), (64, 128), (32, 128), (128, 32))] +
    [("bf16", [1300, 1300], False, 2, 2, 64, 64), ("f32", [600, 3], True, 1, 1, 32, 128), ("f32", [601], False, 1, 1, 128, 32)])


@pytest.mark.parametrize("shape", SCANS, ids=str)
def test_scans(shape):
    x = make(*shape, seed=30, strided=True)
    dtype = shape[0]
    a = (x["q"], x["k"], x["v"], x["g"], x["S0"])
    out, S = gdn().gdn_decay_attn_fwd(*a, scale=x["scale"], cu_seqlens=x["cu_dev"])
    grads = gdn().gdn_decay_attn_bwd(*a, x["do"], x["dS"], scale=x["scale"], cu_seqlens=x["cu_dev"])
    gdn().check_device_status()
    b = [f64(t) for t in a[:4]]
    want, Sw = od.forward(*b, f64(x["S0"]), x["scale"], x["cu"])
    close(want, out, TOL[dtype], "out")
    close(Sw, S, STATE_TOL, "S_final")
    gw = od.backward(*b, f64(x["do"]), f64(x["S0"]), f64(x["dS"]), x["scale"], x["cu"])
    for name, w, g in zip(("grad_q", "grad_k", "grad_v"), gw, grads):
        close(w, g, TOL[dtype], name)
    close(gw[3], grads[3], STATE_TOL, "grad_S0")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,Hqk,Hv,dk,dv", [(40, 8, 16, 128, 128), (40, 16, 16, 64, 128), (160, 2, 4, 32, 32),
                                            (160, 4, 4, 64, 64), (160, 1, 4, 32, 128), (160, 4, 4, 128, 32)])
@pytest.mark.parametrize("pooled", [False, True])
def test_steps_of_whole_states(dtype, N, Hqk, Hv, dk, dv, pooled):
    x = make(dtype, [1] * N, False, Hqk, Hv, dk, dv, seed=31, strided=True)
    q, k, v = (x[n][:, 0] for n in "qkv")
    S, slots = x["S0"], None
    gen = torch.Generator().manual_seed(1)
    if pooled:
        S = torch.randn(N + 9, Hv, dk, dv, generator=gen).cuda()
        slots = torch.randperm(N + 9, generator=gen)[:N].to(torch.int32)
        slots[::5] = -1
    want, Sw = od.step(f64(q), f64(k), f64(v), f64(x["g"]), f64(S), None if slots is None else slots.tolist(), 0.25)
    out = gdn().gdn_decay_attn_step(q, k, v, x["g"], S, slots=None if slots is None else slots.cuda(), scale=0.25)
    close(want, out, TOL[dtype] if dtype == "f32" else 2.0 ** -8, "out")
    close(Sw, S, 1e-6, "S")


@pytest.mark.parametrize("case", [("f32", 400, 8192, 2, True), ("f32", 500, 4840, 2, True), ("f32", 400, 8192, 1, False),
                                  ("f32", 330, 7256, 2, False), ("bf16", 500, 8192, 2, True)], ids=str)
def test_norms_with_few_stages_over_many_rows(case):
    bn.test_forward_and_backward(case)


def captured(call, change):
    """call's results from a CUDA graph replayed after `change`, and the call's own then."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()   # first use of its kernels
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = call()
    change()
    graph.replay()
    got = [None if t is None else t.clone() for t in res]
    return got, call()


@pytest.mark.parametrize("name", ["fwd", "fwd segments", "bwd", "step", "norm", "norm bwd"])
def test_a_captured_call_replays_on_other_inputs(name):
    lens, packed, dtype = ([1400, 3], True, "bf16") if name == "fwd segments" else ([90, 90], False, "bf16")
    x = make(dtype, lens, packed, 2, 4, 64, 64, seed=32)
    y = bn.make("bf16", 70, 512, 2, True, seed=33)
    q, k, v, g, S0 = (x[n] for n in ("q", "k", "v", "g", "S0"))
    if name.startswith("fwd"):
        call = lambda: gdn().gdn_decay_attn_fwd(q, k, v, g, S0, cu_seqlens=x["cu_dev"])   # noqa: E731
    elif name == "bwd":
        call = lambda: gdn().gdn_decay_attn_bwd(q, k, v, g, S0, x["do"], x["dS"])   # noqa: E731
    elif name == "step":
        pool = S0.clone()

        def call():
            pool.copy_(S0)
            return gdn().gdn_decay_attn_step(q[:, 0], k[:, 0], v[:, 0], g, pool), pool
    else:
        a, kw = (y["x"], y["b"], y["wa"], y["wb"]), dict(gate=y["gate"], res_scale=y["c"])
        call = ((lambda: gdn().gdn_block_norm_fwd(*a, **kw)) if name == "norm" else
                (lambda: gdn().gdn_block_norm_bwd(*a, y["gr"], y["gn"], **kw)))

    def change():
        for t in (q, k, v, S0, x["do"], x["dS"], y["x"], y["b"], y["gate"], y["gr"]):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(t.numel())))
        g.mul_(0.5)

    got, want = captured(call, change)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
