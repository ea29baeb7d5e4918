"""The selective scan's and the layer norm's entry points on the host: what they refuse before anything is launched, their
workspaces, and which layouts of rows the binding takes (no call here reaches a kernel)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
L = pytest.importorskip("gated_deltanet_recurrence_03_gb300._lib")
from gated_deltanet_recurrence_03_gb300 import api   # noqa: E402

FAKE = 0x10000   # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_recurrence_03_gb300 import build
    build.build()
    return L.load()


def opts(lib, **kw):
    o = L.default_opts(lib)
    for k, v in kw.items():
        setattr(o, k, v)
    return ctypes.byref(o)


def scan(lib, what="fwd", B=1, T=8, D=16, G=1, N=16, strides=(0, 0, 0, 0, 0), ptrs=(), slots=FAKE, num_slots=1, g=(0, 0, 0), **kw):
    p = {n: FAKE for n in ("u", "delta", "A_log", "B", "C", "skip", "dt_bias", "z", "h0", "y", "hf", "gy", "gh", "gu", "gd", "gA",
                           "gB", "gC", "gs", "gb", "gz", "gh0")} | dict(ptrs)
    head = (p["u"], strides[0], p["delta"], strides[1], p["A_log"], p["B"], strides[2], p["C"], strides[3], p["skip"],
            p["dt_bias"], p["z"], strides[4])
    if what == "fwd":
        return lib.gdn_selective_scan_fwd(*head, p["h0"], p["y"], p["hf"], B, T, D, G, N, opts(lib, **kw))
    if what == "step":
        return lib.gdn_selective_scan_step(*head, p["h0"], slots, num_slots, p["y"], T, D, G, N, opts(lib, **kw))
    return lib.gdn_selective_scan_bwd(*head, p["h0"], p["gy"], p["gh"], p["gu"], p["gd"], p["gA"], p["gB"], g[0], p["gC"], g[1],
                                      p["gs"], p["gb"], p["gz"], g[2], p["gh0"], B, T, D, G, N, opts(lib, **kw))


ARG, UNSUPPORTED, WORKSPACE = L.GDN_ERR_INVALID_ARG, L.GDN_ERR_UNSUPPORTED, L.GDN_ERR_WORKSPACE
COMMON = [(dict(T=-1), ARG), (dict(D=0), ARG), (dict(D=20), ARG), (dict(D=16, G=3), ARG), (dict(D=24, G=2), ARG), (dict(G=0), ARG),
          (dict(N=12), UNSUPPORTED), (dict(N=128), UNSUPPORTED), (dict(dtype=5), ARG), (dict(flags=1), ARG),
          (dict(num_events=1), ARG), (dict(strides=(8, 0, 0, 0, 0)), ARG), (dict(strides=(0, 20, 0, 0, 0)), ARG),
          (dict(strides=(0, 0, 8, 0, 0)), ARG), (dict(strides=(0, 0, 0, 2 ** 31, 0)), ARG), (dict(strides=(0, 0, 0, 0, -16)), ARG),
          (dict(ptrs={"u": 0}), ARG), (dict(ptrs={"delta": 0}), ARG), (dict(ptrs={"A_log": 0}), ARG), (dict(ptrs={"C": 0}), ARG),
          (dict(ptrs={"B": FAKE + 2}), ARG), (dict(ptrs={"z": FAKE + 8}), ARG), (dict(ptrs={"skip": FAKE + 4}), ARG),
          (dict(D=2 ** 27, N=64), ARG)]


@pytest.mark.parametrize("what", ["fwd", "step", "bwd"])
@pytest.mark.parametrize("case,expect", COMMON, ids=str)
def test_common_refusals(lib, what, case, expect):
    assert scan(lib, what, **case) == expect
    assert lib.gdn_last_error() != b""


@pytest.mark.parametrize("what", ["fwd", "bwd"])
@pytest.mark.parametrize("case", [dict(B=-1), dict(B=2, cu_seqlens=FAKE, num_seqs=2), dict(cu_seqlens=FAKE, num_seqs=0),
                                  dict(cu_seqlens=FAKE + 2, num_seqs=1), dict(B=2 ** 16, T=2 ** 16),
                                  dict(D=4096, cu_seqlens=FAKE, num_seqs=2 ** 30), dict(T=2 ** 30, D=2 ** 12, G=2 ** 9)], ids=str)
def test_sequence_refusals(lib, what, case):
    assert scan(lib, what, **case) == ARG
    assert lib.gdn_last_error() != b""


def test_other_refusals(lib):
    assert scan(lib, "fwd", ptrs={"y": 0}) == ARG and scan(lib, "fwd", ptrs={"h0": FAKE + 4}) == ARG
    assert scan(lib, "step", slots=0, num_slots=7) == ARG and scan(lib, "step", num_slots=-1) == ARG
    assert scan(lib, "step", slots=FAKE + 2) == ARG and scan(lib, "step", ptrs={"h0": 0}) == ARG
    assert scan(lib, "step", T=2 ** 24, D=2 ** 16, num_slots=2 ** 24) == ARG
    for n in ("gy", "gu", "gd", "gB", "gC", "gz"):
        assert scan(lib, "bwd", ptrs={n: 0}) == ARG
        assert scan(lib, "bwd", ptrs={n: FAKE + 4}) == ARG
    for g in ((8, 0, 0), (0, 20, 0), (0, 0, 8)):
        assert scan(lib, "bwd", g=g) == ARG
    assert scan(lib, "bwd") == WORKSPACE   # none given
    assert scan(lib, "bwd", workspace=FAKE, workspace_bytes=16) == WORKSPACE
    assert scan(lib, "bwd", workspace=FAKE + 16, workspace_bytes=1 << 40) == ARG
    assert scan(lib, "fwd", T=4096) == WORKSPACE   # few channels, many tokens: segments


def test_nothing_to_do(lib):
    empty = {n: 0 for n in ("u", "delta", "B", "C", "y", "h0", "hf", "z", "gy", "gu", "gd", "gB", "gC", "gz", "gh", "gh0", "gA", "gs",
                            "gb")}
    for what in ("fwd", "bwd"):
        assert scan(lib, what, B=0, ptrs=empty) == L.GDN_OK
    assert scan(lib, "step", T=0, slots=0, ptrs=empty) == L.GDN_OK


def test_workspace_queries(lib):
    f, b = lib.gdn_selective_scan_fwd_workspace_size, lib.gdn_selective_scan_bwd_workspace_size
    assert f(2, 8192, 4096, 1, 16, opts(lib)) < b(2, 8192, 4096, 1, 16, opts(lib))
    assert f(1, 50, 64, 1, 16, opts(lib)) == 0   # one segment
    assert f(1, 50000, 64, 1, 16, opts(lib)) >= 50000 // 4096 * 64 * 17 * 4
    for bad in ((0, 8, 16, 1, 16), (1, 0, 16, 1, 16), (1, 8, 12, 1, 16), (1, 8, 16, 0, 16), (1, 8, 16, 1, 7), (-1, 8, 16, 1, 16)):
        assert f(*bad, opts(lib)) == 0 and b(*bad, opts(lib)) == 0
    assert f(1, 8, 16, 1, 16, opts(lib, cu_seqlens=FAKE, num_seqs=-3)) == 0
    assert b(1, 8, 16, 1, 16, opts(lib, cu_seqlens=FAKE, num_seqs=0)) == 0


def norm(lib, what="fwd", rows=2, D=16, ptrs=(), **kw):
    p = {n: FAKE for n in ("x", "b", "w", "bias", "n", "gn", "gr", "gx", "gw", "gb")} | {"r": FAKE + 256} | dict(ptrs)
    if what == "fwd":
        return lib.gdn_layer_norm_fwd(p["x"], p["b"], p["w"], p["bias"], p["n"], p["r"], rows, D, opts(lib, **kw))
    return lib.gdn_layer_norm_bwd(p["x"], p["b"], p["w"], p["gn"], p["gr"], p["gx"], p["gw"], p["gb"], rows, D, opts(lib, **kw))


@pytest.mark.parametrize("case,expect", [
    (dict(rows=-1), ARG), (dict(rows=2 ** 31), ARG), (dict(D=12), ARG), (dict(D=0), ARG), (dict(D=8200), UNSUPPORTED),
    (dict(dtype=9), ARG), (dict(flags=4), ARG), (dict(norm_eps=-1.0), ARG), (dict(norm_eps=float("nan")), ARG),
    (dict(num_events=-1), ARG), (dict(ptrs={"x": 0}), ARG), (dict(ptrs={"w": 0}), ARG), (dict(ptrs={"x": FAKE + 8}), ARG),
    (dict(ptrs={"b": FAKE + 2}), ARG), (dict(ptrs={"w": FAKE + 4}), ARG)], ids=str)
@pytest.mark.parametrize("what", ["fwd", "bwd"])
def test_norm_refusals(lib, what, case, expect):
    assert norm(lib, what, **case) == expect
    assert lib.gdn_last_error() != b""


def test_norm_pairs_workspace_and_no_rows(lib):
    assert norm(lib, ptrs={"r": 0}) == ARG and norm(lib, ptrs={"b": 0}) == ARG and norm(lib, ptrs={"r": FAKE}) == ARG
    assert norm(lib, ptrs={"n": 0}) == ARG
    for n in ("gn", "gx"):
        assert norm(lib, "bwd", ptrs={n: 0}) == ARG
    assert norm(lib, "bwd") == WORKSPACE
    assert norm(lib, rows=0) == L.GDN_OK
    assert norm(lib, "bwd", rows=0, ptrs={"gw": 0, "gb": 0}) == L.GDN_OK
    assert lib.gdn_layer_norm_bwd_workspace_size(10, 64, opts(lib)) == 10 * 2 * 64 * 4
    assert lib.gdn_layer_norm_bwd_workspace_size(10, 12, opts(lib)) == 0


@pytest.mark.parametrize("t,lead,row", [
    (torch.zeros(2, 5, 24), 2, 24), (torch.zeros(2, 5, 48)[..., 24:], 2, 48), (torch.zeros(2, 5, 48)[:, :1, :24], 2, 240),
    (torch.zeros(1, 1, 8).expand(1, 1, 8), 2, 8), (torch.zeros(7, 24), 1, 24), (torch.zeros(7, 2, 24)[:, 1], 1, 48),
    (torch.zeros(2, 5, 40)[..., 8:24].unflatten(-1, (2, 8)), 2, 40), (torch.zeros(2, 0, 24), 2, 24)],
    ids=lambda x: str(getattr(x, "shape", x)))
def test_rows_taken(t, lead, row):
    width = int(torch.tensor(t.shape[lead:]).prod())
    assert api._row_stride("x", t, lead, width) == row


@pytest.mark.parametrize("t,lead", [
    (torch.zeros(1, 1, 24).expand(1, 6, 24), 2), (torch.zeros(1, 1, 24).expand(4, 1, 24), 2), (torch.zeros(1, 24).expand(5, 24), 1),
    (torch.zeros(1, 6, 24).expand(4, 6, 24), 2), (torch.zeros(24, 6).t(), 1), (torch.zeros(1, 6, 48)[..., ::2], 2),
    (torch.zeros(300).as_strided((1, 6, 24), (300, 8, 1)), 2), (torch.zeros(6, 2, 16)[..., :8], 1)],
    ids=lambda x: str(getattr(x, "shape", x)))
def test_rows_refused(t, lead):
    width = int(torch.tensor(t.shape[lead:]).prod())
    with pytest.raises(ValueError, match="rows"):
        api._row_stride("x", t, lead, width)


def test_binding_refuses_wrong_tensors():
    u, A, B = torch.zeros(1, 4, 16), torch.zeros(16, 8), torch.zeros(1, 4, 1, 8)
    for args in ((u[0], u, A, B, B), (u, u, A[0], B, B), (u, u, A, B[..., 0], B), (u, u[:, :2], A, B, B), (u, u.bfloat16(), A, B, B),
                 (u.half(), u.half(), A, B.half(), B.half()), (u, u, A, B, B[..., :4]), (u, u, A.double(), B, B)):
        with pytest.raises(ValueError):
            api.gdn_selective_scan_fwd(*args)
    for args in ((None, u, A, B, B), (u, None, A, B, B), (u, u, None, B, B), (u, u, A, None, B), (u, u, A, B, 3)):
        with pytest.raises(TypeError):
            api.gdn_selective_scan_fwd(*args)
    every = u[:, :1].expand(1, 4, 16)
    with pytest.raises(ValueError, match="rows"):
        api.gdn_selective_scan_fwd(every, u, A, B, B)
    with pytest.raises(ValueError):
        api.gdn_selective_scan_step(u[0], u[0], A, B[0], B[0], torch.zeros(3, 16, 8))   # three states for four rows


@pytest.mark.parametrize("i", range(5))
def test_strides_up_to_two_to_the_24(lib, i):
    """What a kernel steps over at once stays within 32 bits: a longer stride is refused, the longest one is not."""
    at = lambda v: tuple(v if j == i else 0 for j in range(5))   # noqa: E731
    for what in ("fwd", "step", "bwd"):
        assert scan(lib, what, strides=at(2 ** 24 + 8)) == ARG
        # past the strides' check: refused for what comes behind it
        assert scan(lib, what, strides=at(2 ** 24), ptrs={"A_log": FAKE + 4}) == ARG and b"stride" not in lib.gdn_last_error()
    if i >= 2:
        g = tuple(2 ** 24 + 8 if j == i - 2 else 0 for j in range(3))
        assert scan(lib, "bwd", g=g) == ARG and b"stride" in lib.gdn_last_error()
