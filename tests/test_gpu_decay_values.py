"""GPU: decays that are not ordinary ones: growths, infinities, values whose powers overflow, NaN.  They stay in their
head, a call with them ends, and what the formula makes NaN is NaN."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import decay as od   # noqa: E402
from test_gpu_decay_attn import STATE_TOL, TOL, close, f64, gdn, make   # noqa: E402

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

SHAPES = [("bf16", [300], False, 128), ("bf16", [77, 0, 140], True, 64), ("f32", [70, 1, 33], True, 64),
          ("bf16", [1300], False, 128)]   # (the last in segments)


def calls(x, g, scale=0.1):
    a = (x["q"], x["k"], x["v"], g, x["S0"])
    res = (*gdn().gdn_decay_attn_fwd(*a, scale=scale, cu_seqlens=x["cu_dev"]),
           *gdn().gdn_decay_attn_bwd(*a, x["do"], x["dS"], scale=scale, cu_seqlens=x["cu_dev"]))
    pool = x["S0"].clone()
    n = len(pool)
    step = gdn().gdn_decay_attn_step(*(x[m][0, :n] for m in "qkv"), g, pool, scale=scale)
    gdn().check_device_status()
    names = ("out", "S_final", "grad_q", "grad_k", "grad_v", "grad_S0")
    return dict(zip(names, res)) | {"step": step, "pool": pool}


def head(name, t, h):
    return t[:, h] if name in ("S_final", "grad_S0", "step", "pool") else t[:, :, h]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_decays_without_bound_end_and_stay_in_their_head(shape):
    dtype, lens, packed, d = shape
    x = make(dtype, lens, packed, 4, 4, d, d, seed=20)
    g = torch.tensor([-0.1, -0.3, -0.01, -0.2]).cuda()
    clean = calls(x, g)
    g[1], g[3] = float("inf"), 3e38
    odd = calls(x, g)
    for name, t in odd.items():
        for h in (0, 2):
            assert torch.equal(head(name, t, h), head(name, clean[name], h)), (name, h)
    for name in ("out", "S_final", "grad_S0"):
        for h in (1, 3):
            assert not torch.isfinite(head(name, odd[name], h)).all(), (name, h)


@pytest.mark.parametrize("shape", SHAPES[:3], ids=str)
def test_growths_follow_the_formula(shape):
    """exp(0.004 * 300) to exp(0.03 * 300), per head; tolerances as for decays."""
    dtype, lens, packed, d = shape
    x = make(dtype, lens, packed, 2, 2, d, d, seed=21)
    g = torch.tensor([0.004, 0.03]).cuda()
    got = calls(x, g)
    a = [f64(x[n]) for n in "qkv"] + [f64(g)]
    out, S = od.forward(*a, f64(x["S0"]), 0.1, x["cu"])
    gq, gk, gv, gS = od.backward(*a, f64(x["do"]), f64(x["S0"]), f64(x["dS"]), 0.1, x["cu"])
    for name, want in (("out", out), ("grad_q", gq), ("grad_k", gk), ("grad_v", gv), ("S_final", S), ("grad_S0", gS)):
        for h in range(2):
            close(head(name, want, h), head(name, got[name], h), STATE_TOL if "S" in name else TOL[dtype], (name, h))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_nan_decay_shows(shape):
    """Everything that a NaN decay multiplies is NaN, in its head only; the gradients of a sequence's last token see no
    decay and are finite, and sequences without tokens keep their states."""
    dtype, lens, packed, d = shape
    x = make(dtype, lens, packed, 3, 3, d, d, seed=22)
    g = torch.tensor([-0.1, -0.3, -0.01]).cuda()
    clean = calls(x, g)
    g[1] = float("nan")
    got = calls(x, g)
    a = [f64(x[n]) for n in "qkv"] + [f64(g)]
    out, S = od.forward(*a, f64(x["S0"]), 0.1, x["cu"])
    gq, gk, gv, gS = od.backward(*a, f64(x["do"]), f64(x["S0"]), f64(x["dS"]), 0.1, x["cu"])
    want = {"out": out, "S_final": S, "grad_q": gq, "grad_k": gk, "grad_v": gv, "grad_S0": gS}
    n = len(lens)
    want["step"], want["pool"] = od.step(*(f64(x[m][0, :n]) for m in "qkv"), f64(g), f64(x["S0"]), scale=0.1)
    for name, w in want.items():
        for h in (0, 2):
            assert torch.equal(head(name, got[name], h), head(name, clean[name], h)), (name, h)
        assert np.array_equal(np.isnan(head(name, w, 1)), np.isnan(f64(head(name, got[name], 1)))), name
