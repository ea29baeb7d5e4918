"""GPU: a value of the selective scan's inputs that is not finite reaches only what the formula gives it to: everything else
is, bit for bit, what it is without that value."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gated_deltanet_recurrence_03_gb300 as gdn  # noqa: E402

B, T, D, G, N = 2, 150, 80, 2, 16
T0, D0, N0 = 70, 5, 3            # where the value is: sequence 0, token T0, channel D0 of group 0, state N0
NAMES = ("y", "h", "u", "delta", "A_log", "B", "C", "skip", "dt_bias", "z", "h0")


def inputs(dtype):
    gen = torch.Generator().manual_seed(11)
    r = lambda *s, dt=dtype: torch.randn(*s, generator=gen).cuda().to(dt)   # noqa: E731
    f32 = torch.float32
    return dict(u=r(B, T, D), delta=r(B, T, D), A_log=r(D, N, dt=f32), B=r(B, T, G, N), C=r(B, T, G, N), skip=r(D, dt=f32),
                dt_bias=r(D, dt=f32), z=r(B, T, D), h0=r(B, D, N, dt=f32), gy=r(B, T, D), gh=r(B, D, N, dt=f32))


def run(x):
    kw = dict(skip=x["skip"], dt_bias=x["dt_bias"], z=x["z"])
    main = x["u"], x["delta"], x["A_log"], x["B"], x["C"], x["h0"]
    return dict(zip(NAMES, (*gdn.gdn_selective_scan_fwd(*main, **kw), *gdn.gdn_selective_scan_bwd(*main, x["gy"], x["gh"], **kw))))


def reached(what):
    """Masks of what may change."""
    m = {k: torch.zeros(s, dtype=torch.bool) for k, s in dict(
        y=(B, T, D), h=(B, D, N), u=(B, T, D), delta=(B, T, D), A_log=(D, N), B=(B, T, G, N), C=(B, T, G, N), skip=(D,),
        dt_bias=(D,), z=(B, T, D), h0=(B, D, N)).items()}
    group = slice(0, D // G)
    if what == "B":       # h of the group's channels from T0 on: q of that token alone, w of the later ones
        m["y"][0, T0:, group] = m["z"][0, T0:, group] = m["delta"][0, T0:, group] = True
        m["u"][0, T0, group] = m["dt_bias"][group] = True
        m["C"][0, T0:, 0, N0] = m["h"][0, group, N0] = m["A_log"][group, N0] = True
    elif what == "C":     # y of that token, lam of the tokens up to it
        m["y"][0, T0, group] = m["z"][0, T0, group] = True
        m["u"][0, :T0 + 1, group] = m["delta"][0, :T0 + 1, group] = m["dt_bias"][group] = True
        m["B"][0, :T0 + 1, 0, N0] = m["A_log"][group, N0] = m["h0"][0, group, N0] = True
    elif what == "gy":    # p of one channel's token
        m["u"][0, :T0 + 1, D0] = m["delta"][0, :T0 + 1, D0] = m["z"][0, T0, D0] = True
        m["B"][0, :T0 + 1, 0] = m["C"][0, T0, 0] = True
        m["A_log"][D0] = m["skip"][D0] = m["dt_bias"][D0] = m["h0"][0, D0] = True
    elif what == "h0":    # one state of one channel
        m["y"][0, :, D0] = m["z"][0, :, D0] = m["delta"][0, :, D0] = m["dt_bias"][D0] = True
        m["h"][0, D0, N0] = m["A_log"][D0, N0] = m["C"][0, :, 0, N0] = True
    else:                 # gh: one state's lam
        m["u"][0, :, D0] = m["delta"][0, :, D0] = m["dt_bias"][D0] = True
        m["B"][0, :, 0, N0] = m["A_log"][D0, N0] = m["h0"][0, D0, N0] = True
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["B", "C", "gy", "h0", "gh"])
def test_what_is_not_finite_goes_no_further_than_the_formula(what, value, dtype):
    x = inputs(dtype)
    want = run(x)
    at = {"B": (0, T0, 0, N0), "C": (0, T0, 0, N0), "gy": (0, T0, D0)}.get(what, (0, D0, N0))
    x[what][at] = value
    got = run(x)
    for name, mask in reached(what).items():
        clean = ~mask.cuda()
        assert torch.equal(got[name][clean], want[name][clean]), name
    # and it does reach the first results it belongs to
    key, where = {"B": ("y", (0, T0, 0)), "C": ("y", (0, T0, 0)), "gy": ("u", (0, T0, D0)), "h0": ("y", (0, 0, D0)),
                  "gh": ("u", (0, T - 1, D0))}[what]
    assert not torch.isfinite(got[key][where])
