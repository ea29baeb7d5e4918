"""The decay over n tokens in two floats, exp(g n) = hi + lo (csrc/decay_unit.cuh), on the host and on the device.

Bound of the relative error, for x = g n in [-12, 12] with s halvings to |x| / 2^s <= 2^-10 (units of one rounding:
2^-24).  The series: its quadratic term is at most 2^-21 with three roundings, 3 * 2^-45 < 2^-43.4, and every squaring
doubles a relative error: 2^(s - 43.4).  A squaring's own roundings are those of el, at most 2^-23 |eh| with three
roundings, and the el^2 left out, together below 2^-45 |eh|; against 1 + eh and doubled by the squarings after it they
sum to less than 2 * 2^-45 exp(|x|) below zero and 2^-45 * 2^s above (s >= 1).  The last rounding of lo adds 2^-47.
In sum below 2^(s - 43) + 2^-44 exp(max(-x, 0)) + 2^-47.  Outside [-12, 12] one float: 2^-22."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

from conftest import ROOT

SRC = os.path.join(ROOT, "tests", "cuda", "decay_power.cu")
LIB = os.path.join(ROOT, "_build", "libdecay_power.so")
HEADER = os.path.join(ROOT, "gated_deltanet_recurrence_03_gb300", "csrc", "decay_unit.cuh")


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_recurrence_03_gb300 import build as b
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(SRC), os.path.getmtime(HEADER)):
        subprocess.check_call([b._nvcc(), *b.NVCC_FLAGS, "-Xcompiler", "-ffp-contract=off", "-shared", "-o", LIB, SRC])
    return LIB


def powers(path, g, n):
    lib = ctypes.CDLL(path)
    g, n = (np.ascontiguousarray(x, np.float32) for x in (g, n))
    hi, lo = np.zeros_like(g), np.zeros_like(g)
    f = ctypes.POINTER(ctypes.c_float)
    lib.decay_power_host(*(x.ctypes.data_as(f) for x in (g, n, hi, lo)), ctypes.c_int(g.size))
    return hi.astype(np.float64), lo.astype(np.float64)


def device_powers(path, g, n):
    import torch
    lib = ctypes.CDLL(path)
    lib.decay_power_device.argtypes = [ctypes.c_void_p] * 4 + [ctypes.c_int]
    g, n = (torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda() for x in (g, n))
    hi, lo = torch.zeros_like(g), torch.zeros_like(g)
    assert lib.decay_power_device(g.data_ptr(), n.data_ptr(), hi.data_ptr(), lo.data_ptr(), g.numel()) == 0
    return hi.double().cpu().numpy(), lo.double().cpu().numpy()


@pytest.mark.parametrize("run", [powers, pytest.param(device_powers, marks=pytest.mark.gpu)], ids=["host", "device"])
def test_accuracy_against_64_bits(lib, run):
    rng = np.random.default_rng(0)
    g = np.concatenate([-np.exp2(-rng.uniform(-2, 24, 20000)), np.exp2(-rng.uniform(3, 24, 2000)), [0.0, -0.0, -0.09375]])
    n = np.concatenate([rng.integers(1, 129, 22000), [128, 1, 128]])
    g = g.astype(np.float32)
    x = g.astype(np.float64) * n   # exact: 24 bits times 8
    hi, lo = run(lib, g, n)
    err = np.abs((hi + lo) / np.exp(x) - 1.0)
    s = np.maximum(np.ceil(np.log2(np.maximum(np.abs(x), 1e-300))) + 10, 0)
    inside = np.abs(x) <= 12
    bound = np.exp2(s - 43) + 2.0 ** -44 * np.exp(np.maximum(-x, 0)) + 2.0 ** -47
    assert (err[inside] <= bound[inside]).all(), (err / bound)[inside].max()
    far = (x < -12) & (x > -80)   # (below that the result is no longer a normal number)
    assert inside.sum() > 1000 and far.sum() > 100 and (err[far] <= 2.0 ** -22).all()
    assert (np.abs(lo) <= 2.0 ** -24 * hi + 1e-45).all()


def test_every_value_ends(lib):
    """Infinities, values whose product with n overflows, and NaN, in a process of its own with a time limit."""
    code = (f"import sys; sys.path.insert(0, {os.path.dirname(__file__)!r}); import numpy as np; from test_decay_power import powers\n"
            "g = np.array([np.inf, 3e38, 1e36, 1.0, -np.inf, -3e38, np.nan], np.float32)\n"
            f"hi, lo = powers({lib!r}, g, np.full(7, 128))\n"
            "assert np.isinf(hi[:4]).all() and (hi[4:6] == 0).all() and np.isnan(hi[6]) and (lo[:6] == 0).all()\n")
    r = subprocess.run([sys.executable, "-c", code], timeout=60, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
