"""GPU: decays that are not ordinary ones: growths, infinities, values whose powers overflow, NaN.  They stay in their
head, a call with them ends, and what the formula makes NaN is NaN.  Inputs that are not finite reach what the formula
gives them to, and nothing else."""
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


PLACES = ("first", "inside", "last")


@pytest.mark.parametrize("shape", [("bf16", [300], False, 128), ("bf16", [77, 0, 140], True, 64),
                                   ("bf16", [1300], False, 32), ("f32", [70, 1, 33], True, 64),
                                   ("f32", [200], False, 128)], ids=str)
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
@pytest.mark.parametrize("value", [float("nan"), -float("inf")], ids=["nan", "inf"])
def test_a_value_that_is_not_finite_reaches_only_what_the_formula_gives_it(shape, which, value):
    """One bad element: results are finite where the formula's are (earlier tokens' outputs, say) and equal there to the
    clean ones; where the formula has NaN they are NaN, and where it has infinities not finite."""
    dtype, lens, packed, d = shape
    x = make(dtype, lens, packed, 1, 2, d, d, seed=23)
    g = torch.tensor([-0.05, -0.3]).cuda()
    clean = calls(x, g)
    total = sum(lens)
    for place in PLACES:
        t = {"first": 0, "inside": min(lens[0] - 2, 45), "last": total - 1}[place]
        y = dict(x)
        y[which] = x[which].clone()
        y[which][0, t, -1, 5] = value
        got = calls(y, g)
        a = [f64(y[n]) for n in "qkv"] + [f64(g)]
        with np.errstate(invalid="ignore"):
            out, S = od.forward(*a, f64(x["S0"]), 0.1, x["cu"])
            gq, gk, gv, gS = od.backward(*a, f64(y["do"]), f64(x["S0"]), f64(x["dS"]), 0.1, x["cu"])
        for name, want in (("out", out), ("S_final", S), ("grad_q", gq), ("grad_k", gk), ("grad_v", gv), ("grad_S0", gS)):
            have, fine = f64(got[name]), np.isfinite(want)
            assert np.array_equal(np.isfinite(have), fine), (place, name)
            assert np.array_equal(have[fine], f64(clean[name])[fine]), (place, name)
            if np.isnan(value):
                assert np.array_equal(np.isnan(have), np.isnan(want)), (place, name)
