"""GPU: a value that is not finite in a sequence's last token, where the gradients' walk goes on to the end of its chunk of
eight tokens.  The formula gives the state behind the last token to h_final, y and dC alone: dA_log takes h_{t-1}, so that it
keeps every bit, as does all else that the value does not enter."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gated_deltanet_recurrence_03_gb300 as gdn  # noqa: E402

LENS = (1, 7, 8, 9, 41, 64, 700)   # less than a chunk, a whole one, one more; several segments
D, G, D0, N0 = 80, 2, 5, 3         # the value's channel (group 0) and state
NAMES = ("y", "h", "u", "delta", "A_log", "B", "C", "skip", "dt_bias", "z", "h0")


def inputs(dtype, N):
    gen = torch.Generator().manual_seed(12)
    T, n, f32 = sum(LENS), len(LENS), torch.float32
    r = lambda *s, dt=dtype: torch.randn(*s, generator=gen).cuda().to(dt)   # noqa: E731
    cu = torch.tensor([sum(LENS[:i]) for i in range(n + 1)], dtype=torch.int32).cuda()
    return dict(u=r(1, T, D), delta=r(1, T, D), A_log=r(D, N, dt=f32), B=r(1, T, G, N), C=r(1, T, G, N), skip=r(D, dt=f32),
                dt_bias=r(D, dt=f32), z=r(1, T, D), h0=r(n, D, N, dt=f32), gy=r(1, T, D), gh=r(n, D, N, dt=f32), cu=cu)


def run(x):
    kw = dict(skip=x["skip"], dt_bias=x["dt_bias"], z=x["z"], cu_seqlens=x["cu"])
    main = x["u"], x["delta"], x["A_log"], x["B"], x["C"], x["h0"]
    return dict(zip(NAMES, (*gdn.gdn_selective_scan_fwd(*main, **kw), *gdn.gdn_selective_scan_bwd(*main, x["gy"], x["gh"], **kw))))


def reached(what, i, N):
    """Masks of what may change for a value in the last token of sequence i (what = "A_log": in the rate of one state, whose
    decay enters every lam but the last token's)."""
    T, n = sum(LENS), len(LENS)
    t0, e = sum(LENS[:i]), sum(LENS[:i + 1]) - 1
    m = {k: torch.zeros(s, dtype=torch.bool) for k, s in dict(
        y=(1, T, D), h=(n, D, N), u=(1, T, D), delta=(1, T, D), A_log=(D, N), B=(1, T, G, N), C=(1, T, G, N), skip=(D,),
        dt_bias=(D,), z=(1, T, D), h0=(n, D, N)).items()}
    group = slice(0, D // G)
    if what == "B":
        for k in ("y", "z", "u", "delta"):
            m[k][0, e, group] = True
        m["dt_bias"][group] = m["h"][i, group, N0] = m["C"][0, e, 0, N0] = True
    elif what == "u":
        for k in ("y", "z", "delta"):
            m[k][0, e, D0] = True
        m["dt_bias"][D0] = m["skip"][D0] = m["h"][i, D0] = True
        m["B"][0, e, 0] = m["C"][0, e, 0] = True
    else:
        for k in ("y", "z", "delta", "u"):
            m[k][0, :, D0] = True
        m["dt_bias"][D0] = m["h"][:, D0, N0] = m["h0"][:, D0, N0] = m["A_log"][D0, N0] = True
        m["B"][0, :, 0, N0] = m["C"][0, :, 0, N0] = True
        for j in range(n):   # the last token of a sequence: lam before any decay
            last = sum(LENS[:j + 1]) - 1
            m["u"][0, last, D0] = m["B"][0, last, 0, N0] = False
    return m


def check(x, want, what, i, N):
    got = run(x)
    for name, mask in reached(what, i, N).items():
        clean = ~mask.cuda()
        assert torch.equal(got[name][clean], want[name][clean]), (name, i)
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [8, 16, 64])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["B", "u"])
def test_last_token_does_not_reach_the_rates_gradient(what, value, N, dtype):
    x = inputs(dtype, N)
    want = run(x)
    for i in range(len(LENS)):
        e = sum(LENS[:i + 1]) - 1
        at = (0, e, 0, N0) if what == "B" else (0, e, D0)
        keep, x[what] = x[what], x[what].clone()
        x[what][at] = value
        got = check(x, want, what, i, N)
        assert not torch.isfinite(got["h"][i, D0, N0])   # it was there
        x[what] = keep


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [8, 16, 64])
def test_a_rate_that_is_no_number_leaves_the_last_lam_alone(N, dtype):
    x = inputs(dtype, N)
    want = run(x)
    x["A_log"][D0, N0] = float("nan")
    check(x, want, "A_log", 0, N)
