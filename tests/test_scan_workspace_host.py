"""The scan's workspaces on the host: what they hold for many short sequences, and which plan the prompts take."""
import ctypes

import pytest

L = pytest.importorskip("gated_deltanet_recurrence_03_gb300._lib")


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_recurrence_03_gb300 import build
    build.build()
    return L.load()


def need(lib, what, B, T, D, G, N, nseq=0):
    o = L.default_opts(lib)
    if nseq:
        o.cu_seqlens, o.num_seqs = 0x10000, nseq
    return getattr(lib, f"gdn_selective_scan_{what}_workspace_size")(B, T, D, G, N, ctypes.byref(o))


@pytest.mark.parametrize("D,G,N", [(4096, 1, 16), (1024, 2, 64), (520, 1, 8)])
@pytest.mark.parametrize("nseq,length", [(1, 16384), (2, 8192), (256, 64), (2048, 8), (16384, 1), (1024, 64), (4096, 16), (3, 5)])
def test_gradients_workspace_follows_tokens_and_sequences(lib, nseq, length, D, G, N):
    """A state for every 8 tokens and every sequence, three (state, adjoint, sum of dA) and 3 D sums for every segment of 32
    tokens or more and every sequence; 2 N sums for every token and tile of 1024 / N channels; nine arrays, each rounded up to
    256 bytes."""
    tokens = nseq * length
    states = tokens // 8 + nseq + 3 * (tokens // 32 + nseq)
    tiles = G * -(-D // G * N // 1024)
    most = 4 * (D * N * states + D * (tokens // 8 + nseq) + 3 * D * (tokens // 32 + nseq) + 2 * N * tiles * tokens) + 9 * 256
    for got in (need(lib, "bwd", 1, tokens, D, G, N, nseq), need(lib, "bwd", nseq, length, D, G, N)):
        assert 4 * D * N * (tokens // 8) <= got <= most
