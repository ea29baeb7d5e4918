"""GPU: failure detection without a GPU fault: when a bounded wait runs out (the test drops a copy or an arrival) the
kernels' shared pieces end within their limits and set the status; without a failure they do their work."""
import ctypes
import os
import subprocess
import time

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

SRC = os.path.join(ROOT, "tests", "cuda", "giveup.cu")
CSRC = os.path.join(ROOT, "gated_deltanet_recurrence_03_gb300", "csrc")
LIB = os.path.join(ROOT, "_build", "libgiveup.so")
LIMIT = 20_000_000   # 20 ms


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_recurrence_03_gb300 import build as b
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    newest = max(os.path.getmtime(f) for f in (SRC, os.path.join(CSRC, "bulk_ring.cuh"), os.path.join(CSRC, "tc_ptx.cuh")))
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        subprocess.check_call([b._nvcc(), *b.NVCC_FLAGS, "-shared", "-o", LIB, SRC])
    L = ctypes.CDLL(LIB)
    L.giveup_ring.argtypes = [ctypes.c_void_p] * 2 + [ctypes.c_int] * 3 + [ctypes.c_ulonglong] + [ctypes.c_void_p] * 2
    L.giveup_pair.argtypes = [ctypes.c_int] * 2 + [ctypes.c_ulonglong] + [ctypes.c_void_p] * 2
    return L


@pytest.mark.parametrize("stages", [1, 2, 4])
@pytest.mark.parametrize("drop", [-1, 0, 5, 8])
def test_a_ring_whose_copy_never_lands_asks_for_no_more(lib, stages, drop):
    rows = 9
    src = torch.randn(rows, 64, device="cuda")
    dst = torch.zeros_like(src)
    status, result = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.time()
    assert lib.giveup_ring(src.data_ptr(), dst.data_ptr(), rows, stages, drop, LIMIT, status.data_ptr(),
                           result.data_ptr()) == 0
    torch.cuda.synchronize()
    assert time.time() - t0 < 5.0
    if drop < 0:
        assert int(status) == 0 and result.tolist() == [rows, 0] and torch.equal(dst, src)
        return
    assert int(status) == 1 and torch.equal(dst[:drop], src[:drop])
    # what had been asked for when row `drop` was waited for: itself, and with more stages the rows up to
    # stages - 2 ahead (the first ones: all stages)
    asked = max(drop + 1, stages) if drop == 0 or stages == 1 else drop + stages - 1
    assert result.tolist() == [min(rows, asked), 1]


@pytest.mark.parametrize("drop", [-1, 0, 1, 4])
def test_a_pair_of_warps_gives_up_together(lib, drop):
    status, result = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.time()
    assert lib.giveup_pair(5, drop, LIMIT, status.data_ptr(), result.data_ptr()) == 0
    torch.cuda.synchronize()
    assert time.time() - t0 < 5.0
    assert int(status) == (drop >= 0) and result.tolist() == [5 if drop < 0 else drop] * 2
