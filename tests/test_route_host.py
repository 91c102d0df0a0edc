"""CPU check of the router's threshold for sigmoid scores: which 32-bit scores
are looked at again in 64 bits, given the k-th largest.  An expert that must not
be chosen, and a lane past the last expert, has the score -inf, so no threshold
may be -inf; and every score that can reach the k-th must be above it.
"""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from conftest import ROOT

SRC = os.path.join(ROOT, "tests", "csrc", "route_host.cpp")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
LOWEST = float(np.finfo(np.float32).min)


@pytest.fixture(scope="module")
def floor(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("route") / "route_host.so")
    subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-O2", "-std=c++17", "-shared", "-fPIC", SRC, "-o", so],
                   check=True)
    fn = ctypes.CDLL(so).ptgg_host_candidate_floor
    fn.restype, fn.argtypes = ctypes.c_float, [ctypes.c_float]
    return fn


def choose(floor, z, bias, k, lanes):
    """The router's steps for one token over `lanes` slots, of which len(z) are experts."""
    f = np.float32
    ninf = f(-np.inf)
    zz, bb = np.full(lanes, ninf, f), np.zeros(lanes, f)
    zz[: len(z)], bb[: len(z)] = z, bias
    with np.errstate(over="ignore"):
        near = np.where(zz > ninf, f(1) / (f(1) + np.exp(-zz)) + bb, ninf).astype(f)
        exact = (1 / (1 + np.exp(-zz.astype(np.float64))) + bb).astype(f)
    able = [i for i in range(lanes) if near[i] > ninf]
    taken = sorted(able, key=lambda i: (-near[i], i))[:k]
    if len(taken) == k:
        at = f(floor(float(near[taken[-1]])))
        again = [i for i in range(lanes) if near[i] >= at]
        taken = sorted(again, key=lambda i: (-exact[i], i))[:k]
    return taken


@pytest.mark.parametrize("kth", [LOWEST, LOWEST * (1 - 2.0 ** -21), LOWEST / 2, -1e30, -1.0, -0.0, 0.0, 1e-38, 0.5, 1.0,
                                 1e30, -LOWEST])
def test_the_threshold_is_finite_and_low_enough(floor, kth):
    at = floor(kth)
    assert np.isfinite(at) and at <= kth
    # twice what a 32-bit score may be off
    assert at <= max(kth - 2.0 ** -21 * (1 + abs(kth)), LOWEST)


@pytest.mark.parametrize("E,lanes", [(60, 64), (40, 64), (256, 256), (100, 128), (7, 32)])
@pytest.mark.parametrize("mask", [LOWEST, LOWEST * (1 - 2.0 ** -21), -1e30])
def test_experts_masked_by_their_bias(floor, E, lanes, mask):
    """Fewer open experts than are chosen: the lowest of the masked ones follow, never a shut one or a lane past the end."""
    rng = np.random.default_rng(E)
    z = rng.normal(size=E).astype(np.float32)
    bias = np.full(E, mask, np.float32)
    bias[[2, 4, 5]] = 0.01
    z[3], bias[3] = -np.inf, 0.02                        # shut, with an ordinary bias
    got = choose(floor, z, bias, 6, lanes)
    assert sorted(got[:3]) == [2, 4, 5] and got[3:] == [0, 1, 6]
