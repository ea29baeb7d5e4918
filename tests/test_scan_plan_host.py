"""Which plan the scan's prompts take, whole walks or segments (segments need scratch, whole walks none): the one that both
measured times, in the comment at scan_fwd_segment, say is faster by more than 5 %."""
import ctypes

import pytest

L = pytest.importorskip("gated_deltanet_recurrence_03_gb300._lib")


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_recurrence_03_gb300 import build
    build.build()
    return L.load()


def segments(lib, B, T, D, N, dtype="bf16", nseq=0, G=1):
    o = L.default_opts(lib)
    o.dtype = {"bf16": L.GDN_BF16, "f32": L.GDN_F32}[dtype]
    if nseq:
        o.cu_seqlens, o.num_seqs = 0x10000, nseq
    return lib.gdn_selective_scan_fwd_workspace_size(B, T, D, G, N, ctypes.byref(o)) > 0


# batch, tokens, channels, states, type, faster in segments
MEASURED = [
    (1, 8192, 2048, 16, "bf16", True), (1, 8192, 4096, 16, "bf16", True), (1, 8192, 4608, 16, "bf16", True),
    (1, 8192, 5760, 16, "bf16", False), (1, 8192, 6144, 16, "bf16", False), (3, 8192, 2048, 16, "bf16", False),
    (1, 8192, 7168, 16, "bf16", False), (1, 8192, 7936, 16, "bf16", False), (2, 8192, 4096, 16, "bf16", False),
    (2, 8192, 4864, 16, "bf16", False), (2, 8192, 5120, 16, "bf16", True), (2, 8192, 5376, 16, "bf16", True),
    (2, 8192, 6144, 16, "bf16", False), (4, 8192, 4096, 16, "bf16", False), (5, 8192, 4096, 16, "bf16", False),
    (1, 32768, 5120, 16, "bf16", True), (1, 32768, 6144, 16, "bf16", False), (1, 2048, 3584, 16, "bf16", True),
    (1, 2048, 6144, 16, "bf16", False), (1, 1024, 2048, 16, "bf16", True), (1, 1024, 5120, 16, "bf16", False),
    (1, 300, 2048, 16, "bf16", False), (1, 8192, 4096, 16, "f32", True), (1, 8192, 5120, 16, "f32", False),
    (1, 8192, 7936, 16, "f32", False), (2, 8192, 5376, 16, "f32", False), (1, 2048, 3584, 16, "f32", True),
    (1, 2048, 4608, 16, "f32", False), (1, 1024, 2048, 16, "f32", True), (1, 1024, 3584, 16, "f32", False),
    (1, 8192, 10240, 8, "bf16", True), (1, 8192, 14336, 8, "bf16", False), (1, 8192, 9216, 8, "f32", True),
    (1, 8192, 11264, 8, "f32", False), (1, 8192, 2048, 32, "bf16", True), (1, 8192, 3584, 32, "bf16", False),
    (1, 8192, 1024, 64, "bf16", True), (1, 8192, 1792, 64, "bf16", False), (1, 8192, 1024, 64, "f32", True),
    (1, 8192, 1280, 64, "f32", False), (1, 300, 64, 16, "bf16", False), (1, 4096, 64, 16, "f32", True),
]


@pytest.mark.parametrize("case", MEASURED, ids=str)
def test_the_faster_plan_is_taken(lib, case):
    *sizes, want = case
    assert segments(lib, *sizes) == want


@pytest.mark.parametrize("channels,want", [(4096, True), (6144, False), (7168, False), (10240, False)])
def test_packed_sequences_are_taken_as_one(lib, channels, want):
    """Their lengths are on the device.  Past a wave of one sequence's blocks the sequences share waves."""
    for nseq in (1, 4, 16):
        assert segments(lib, 1, 8192, channels, 16, nseq=nseq) == want


def test_groups_count_by_their_tiles(lib):
    """128 groups of 8 channels are 128 blocks, as many as 8192 channels of one group."""
    assert not segments(lib, 1, 8192, 1024, 16, G=128) and segments(lib, 1, 8192, 1024, 16)
