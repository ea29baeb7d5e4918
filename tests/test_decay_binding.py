"""The decayed attention's Python entry points on the host: which layouts of token rows they take, and what they
refuse before the library is called (CPU tensors, nothing is launched)."""
import pytest

torch = pytest.importorskip("torch")
pkg_lib = pytest.importorskip("gated_deltanet_recurrence_03_gb300._lib")
from gated_deltanet_recurrence_03_gb300 import api   # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from gated_deltanet_recurrence_03_gb300 import build
    build.build()


def rows_of(t, lead):
    return api._token_rows("x", t, t.shape[-1], lead)


@pytest.mark.parametrize("t,lead,row", [
    (torch.zeros(2, 5, 3, 8), 2, 24),                                    # dense
    (torch.zeros(2, 5, 40)[..., 8:32].unflatten(-1, (3, 8)), 2, 40),     # a slice of a packed projection
    (torch.zeros(2, 5, 40)[:, :1, :24].unflatten(-1, (3, 8)), 2, 200),   # one token of each sequence
    (torch.zeros(1, 1, 1, 8).expand(1, 1, 1, 8), 2, 8),                  # one token row: any stride is right
    (torch.zeros(7, 3, 8), 1, 24),
    (torch.zeros(7, 4, 24)[:, 1].unflatten(-1, (3, 8)), 1, 96),
    (torch.zeros(2, 0, 3, 8), 2, 24), (torch.zeros(0, 3, 8), 1, 24),     # no tokens
], ids=lambda x: str(getattr(x, "shape", x)))
def test_token_rows_taken(t, lead, row):
    assert rows_of(t, lead) == row


BROADCAST = [
    (torch.zeros(1, 1, 3, 8).expand(1, 6, 3, 8), 2),         # one row for every token
    (torch.zeros(1, 1, 3, 8).expand(4, 6, 3, 8), 2),
    (torch.zeros(1, 1, 3, 8).expand(4, 1, 3, 8), 2),         # one token, one row for every sequence
    (torch.zeros(1, 3, 8).expand(5, 3, 8), 1),
    (torch.zeros(1, 6, 3, 8).expand(4, 6, 3, 8), 2),         # one sequence for all
    (torch.zeros(200).as_strided((1, 6, 3, 8), (200, 8, 8, 1)), 2),   # rows that overlap
]


@pytest.mark.parametrize("t,lead", BROADCAST, ids=lambda x: str(getattr(x, "shape", x)))
def test_rows_that_share_memory_are_refused(t, lead):
    """A row stride of 0 means dense rows to the C entry points, which would read past a broadcast tensor."""
    with pytest.raises(ValueError, match="token rows"):
        rows_of(t, lead)


def test_broadcast_inputs_are_refused_by_the_calls():
    one, v, g = torch.zeros(1, 1, 2, 32), torch.zeros(1, 6, 2, 32), torch.zeros(2)
    every = one.expand(1, 6, 2, 32)
    dense = every.contiguous()
    S = torch.zeros(6, 2, 32, 32)
    for q, k, w in ((every, dense, v), (dense, every, v), (dense, dense, every)):
        with pytest.raises(ValueError, match="token rows"):
            api.gdn_decay_attn_fwd(q, k, w, g)
        with pytest.raises(ValueError, match="token rows"):
            api.gdn_decay_attn_bwd(q, k, w, g, None, v)
        with pytest.raises(ValueError, match="token rows"):
            api.gdn_decay_attn_step(q[0], k[0], w[0], g, S)


def test_workspaces_taken_and_refused():
    like = torch.zeros(2)
    o = pkg_lib.GdnOpts()
    given = torch.empty(300, dtype=torch.uint8)
    assert api._scratch(o, 256, given, like) is given and o.workspace == given.data_ptr() and o.workspace_bytes == 300
    assert api._scratch(o, 0, given, like) is None
    new = api._scratch(o, 1001, given, like)   # too small: a new one
    assert new is not given and new.device == like.device and o.workspace_bytes >= 1001 and o.workspace == new.data_ptr()
    for bad in (torch.empty(300, dtype=torch.uint8, device="meta"),           # of another device
                torch.empty(1, dtype=torch.uint8).expand(300), given[::2]):   # more elements than memory, or not its own
        with pytest.raises(ValueError, match="workspace"):
            api._scratch(o, 100, bad, like)


def test_more_blocks_than_a_grid_holds_are_refused():
    """2^26 + 1 empty or short sequences of 64 heads: the grid's blocks would pass 32 bits and only a few would run."""
    import ctypes
    lib, fake = pkg_lib.load(), 0x10000
    o = pkg_lib.default_opts(lib)
    o.cu_seqlens, o.num_seqs = fake, 2 ** 26 + 1
    dims = (1, 8, 64, 64, 128, 128, ctypes.byref(o))
    assert lib.gdn_decay_attn_fwd(fake, 0, fake, 0, fake, 0, fake, None, fake, None, *dims) == pkg_lib.GDN_ERR_INVALID_ARG
    assert b"sequences" in lib.gdn_last_error()
    assert lib.gdn_decay_attn_bwd(fake, 0, fake, 0, fake, 0, fake, None, fake, None, fake, 0, fake, 0, fake, 0, None,
                                  *dims) == pkg_lib.GDN_ERR_INVALID_ARG
    assert b"sequences" in lib.gdn_last_error()
