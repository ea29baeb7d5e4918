"""The decayed attention's and the block norm's C entry points on the host, without a GPU: bad arguments are
refused before any CUDA call, empty calls do nothing, size queries are pure arithmetic."""
import ctypes

import pytest

pkg_lib = pytest.importorskip("gated_deltanet_recurrence_03_gb300._lib")
BAD, UNSUP, WS, OK = pkg_lib.GDN_ERR_INVALID_ARG, pkg_lib.GDN_ERR_UNSUPPORTED, pkg_lib.GDN_ERR_WORKSPACE, pkg_lib.GDN_OK
FAKE = 0x10000   # an aligned address that is never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_recurrence_03_gb300 import build
    build.build()
    return pkg_lib.load()


def opts(lib, **kw):
    o = pkg_lib.default_opts(lib)
    for k, v in kw.items():
        setattr(o, k, v)
    return ctypes.byref(o)


def fwd(lib, B=1, T=8, Hqk=1, Hv=1, dk=32, dv=32, strides=(0, 0, 0), ptrs=None, **kw):
    q, k, v, g, S0, out, Sf = [FAKE] * 7 if ptrs is None else ptrs
    return lib.gdn_decay_attn_fwd(q, strides[0], k, strides[1], v, strides[2], g, S0, out, Sf, B, T, Hqk, Hv, dk, dv,
                                  opts(lib, **kw))


def bwd(lib, B=1, T=8, Hqk=1, Hv=1, dk=32, dv=32, strides=(0,) * 6, ptrs=None, **kw):
    p = [FAKE] * 11 if ptrs is None else ptrs   # q k v g S0 do dS gq gk gv gS0
    s = strides
    return lib.gdn_decay_attn_bwd(p[0], s[0], p[1], s[1], p[2], s[2], p[3], p[4], p[5], p[6], p[7], s[3], p[8], s[4],
                                  p[9], s[5], p[10], B, T, Hqk, Hv, dk, dv, opts(lib, **kw))


def step(lib, N=2, Hqk=1, Hv=1, dk=32, dv=32, strides=(0, 0, 0), num_slots=4, ptrs=None, **kw):
    q, k, v, g, S, slots, out = [FAKE] * 7 if ptrs is None else ptrs
    return lib.gdn_decay_attn_step(q, strides[0], k, strides[1], v, strides[2], g, S, slots, num_slots, out, N, Hqk, Hv,
                                   dk, dv, opts(lib, **kw))


def without(n, i, value=0):
    p = [FAKE] * n
    p[i] = value
    return p


COMMON = [(dict(Hqk=2, Hv=3), BAD), (dict(Hqk=0), BAD), (dict(dk=48), UNSUP), (dict(dv=256), UNSUP), (dict(dtype=9), BAD),
          (dict(flags=pkg_lib.GDN_NORMALIZE_QK), BAD), (dict(flags=0x80), BAD), (dict(num_events=2), BAD)]
SEQ = [(dict(B=-1), BAD), (dict(T=-1), BAD), (dict(B=2, cu_seqlens=FAKE, num_seqs=2), BAD),
       (dict(cu_seqlens=FAKE, num_seqs=0), BAD), (dict(cu_seqlens=FAKE + 2, num_seqs=1), BAD),
       (dict(B=65536, T=65536), BAD)]


@pytest.mark.parametrize("case,expect", COMMON + SEQ + [
    (dict(strides=(16, 0, 0)), BAD), (dict(strides=(0, 36, 0)), BAD), (dict(strides=(0, 0, -32)), BAD),
    (dict(strides=(0, 0, 2 ** 31)), BAD), (dict(strides=(34, 0, 0), dtype=pkg_lib.GDN_F32), BAD),
    *[(dict(ptrs=without(7, i)), BAD) for i in (0, 1, 2, 3, 5)],
    *[(dict(ptrs=without(7, i, FAKE + 8)), BAD) for i in (0, 1, 2, 4, 5, 6)],
    (dict(ptrs=without(7, 3, FAKE + 2)), BAD),
])
def test_forward_refusals(lib, case, expect):
    assert fwd(lib, **case) == expect and lib.gdn_last_error() != b""


@pytest.mark.parametrize("case,expect", COMMON + SEQ + [
    (dict(strides=(0, 0, 0, 0, 36, 0)), BAD), (dict(strides=(0, 0, 0, 16, 0, 0)), BAD),
    *[(dict(ptrs=without(11, i)), BAD) for i in (0, 1, 2, 3, 5, 7, 8, 9)],
    *[(dict(ptrs=without(11, i, FAKE + 4)), BAD) for i in (4, 5, 6, 7, 10)],
    (dict(Hqk=1, Hv=2), WS), (dict(Hqk=1, Hv=2, workspace=FAKE, workspace_bytes=64), WS),
    (dict(Hqk=1, Hv=2, workspace=FAKE + 16, workspace_bytes=1 << 24), BAD),
])
def test_backward_refusals(lib, case, expect):
    assert bwd(lib, **case) == expect and lib.gdn_last_error() != b""


@pytest.mark.parametrize("case,expect", COMMON + [
    (dict(N=-1), BAD), (dict(num_slots=-1), BAD), (dict(ptrs=without(7, 5), num_slots=1), BAD),
    *[(dict(ptrs=without(7, i)), BAD) for i in (0, 1, 2, 3, 4, 6)], (dict(ptrs=without(7, 5, FAKE + 2)), BAD),
    (dict(ptrs=without(7, 4, FAKE + 4)), BAD), (dict(N=2 ** 28, Hv=64, num_slots=2 ** 28), BAD),
    (dict(strides=(40, 36, 0)), BAD),
])
def test_step_refusals(lib, case, expect):
    assert step(lib, **case) == expect and lib.gdn_last_error() != b""


def norm(lib, back=False, rows=4, D=64, cols=1, ptrs=None, **kw):
    p = [FAKE] * 15 if ptrs is None else ptrs   # x b gate scale post pre | r n | gr gn gx gb ggate gpost gpre gscale
    if not back:
        return lib.gdn_block_norm_fwd(p[0], p[1], p[2], cols, p[3], p[4], p[5], p[6], p[7], rows, D, opts(lib, **kw))
    return lib.gdn_block_norm_bwd(p[0], p[1], p[2], cols, p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11], p[12],
                                  p[13], rows, D, opts(lib, **kw))


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("case,expect", [
    (dict(rows=-1), BAD), (dict(rows=2 ** 31), BAD), (dict(D=0), BAD), (dict(D=60), BAD), (dict(D=8200), UNSUP),
    (dict(cols=2), BAD), (dict(dtype=3), BAD), (dict(flags=1), BAD), (dict(norm_eps=-1.0), BAD),
    *[(dict(ptrs=without(15, i)), BAD) for i in (0, 1, 4, 5, 6, 7)],
    *[(dict(ptrs=without(15, i, FAKE + 8)), BAD) for i in (0, 1, 3, 4, 5, 6, 7)],
    (dict(ptrs=without(15, 2, FAKE + 1)), BAD), (dict(ptrs=without(15, 2, FAKE + 2), cols=64), BAD),
])
def test_block_norm_refusals(lib, back, case, expect):
    assert norm(lib, back, **case) == expect and lib.gdn_last_error() != b""


def test_block_norm_backward_needs_its_buffers(lib):
    assert norm(lib, True, ptrs=without(15, 10)) == BAD        # a gate without grad_gate
    assert norm(lib, True, ptrs=without(15, 8)) == BAD         # grad_x
    assert norm(lib, True) == WS                               # weight sums without scratch
    assert norm(lib, True, workspace=FAKE, workspace_bytes=16) == WS


def test_empty_calls_and_sizes(lib):
    assert fwd(lib, B=0, T=0, ptrs=[0] * 7) == OK and bwd(lib, B=0, T=0, ptrs=[0] * 11) == OK
    assert step(lib, N=0, num_slots=0, ptrs=[0] * 7) == OK
    p = [FAKE] * 15
    p[0] = p[1] = p[6] = p[7] = 0
    assert norm(lib, rows=0, ptrs=p) == OK
    for size in (lib.gdn_decay_attn_fwd_workspace_size, lib.gdn_decay_attn_bwd_workspace_size):
        assert size(-1, 8, 1, 1, 32, 32, opts(lib)) == 0 and size(1, 8, 2, 3, 32, 32, opts(lib)) == 0
        assert size(1, 8, 1, 1, 48, 32, opts(lib)) == 0
    # shared query/key heads: an fp32 part of grad_q and grad_k for each value head
    assert lib.gdn_decay_attn_bwd_workspace_size(1, 100, 1, 2, 64, 64, opts(lib)) >= 2 * 100 * 2 * 64 * 4
    assert lib.gdn_block_norm_bwd_workspace_size(10, 64, opts(lib)) >= 2 * 64 * 4
    assert lib.gdn_block_norm_bwd_workspace_size(10, 60, opts(lib)) == 0
