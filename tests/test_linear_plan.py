"""CPU check of the dense product's planner: whatever tile and cut it chooses, the
parts cover each tile's reduction once and fit the workspace that the call asks
for; and each kind of plan that it can return, for each operator, is among the
sizes at which the GPU tests compare products bit for bit.
"""
import collections
import ctypes
import math
import os
import random
import subprocess

import pytest

import moe_expert_grouped_gemm_amd as ptm
from conftest import ROOT
from test_gpu_linear import DGRAD_TILES, FWD_TILES, SHAPES, WGRAD_TILES
from test_gpu_linear_even import PRODUCTS
from test_gpu_linear_plans import FORWARDS, KINDS

SRC = os.path.join(ROOT, "tests", "csrc", "linear_host.cpp")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FWD, DGRAD, WGRAD = 0, 1, 2
STAGE = 64
FEW, WIDE, NARROW = 0, 1, 4
# rows and columns of the tiles, in the planner's order
TILES = [(16, 16), (256, 256), (128, 128), (64, 128), (64, 32), (128, 128), (64, 128), (32, 128)]
Plan = collections.namedtuple("Plan", "tile splits part whole rest parts tails cuts main cut bytes")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("linear") / "linear_host.so")
    subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-O2", "-std=c++17", "-shared", "-fPIC", SRC, "-o", so],
                   check=True)
    fn = ctypes.CDLL(so).ptgg_host_linear_plan
    fn.restype, fn.argtypes = None, [ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.POINTER(ctypes.c_int64)]

    def of(op, M, N, K):
        out = (ctypes.c_int64 * 11)()
        fn(op, M, N, K, out)
        return Plan(*out)

    return of


def product(op, M, N, K):
    """Rows, columns and reduction of what a call of M, N and K computes."""
    return (M, N, K) if op == FWD else (M, K, N) if op == DGRAD else (N, K, M)


def call(op, M, N, K):
    """And back: the call's M, N and K."""
    return (M, N, K) if op == FWD else (M, K, N) if op == DGRAD else (K, M, N)


def kind(p):
    """What the kernels do differently: the tile, and how its reduction is cut."""
    if p.tile != WIDE:
        return p.tile, "parts" if p.splits > 1 else "whole"
    if not p.rest:
        return p.tile, "whole"
    tails = "no tails" if not p.cut else "whole tails" if p.tails == p.rest else "cut tails" if p.cuts > 1 else "tails"
    return p.tile, tails, "one part" if p.parts == 1 else "parts", "after whole tiles" if p.whole else "alone"


def sizes(rng, op):
    """Sizes that the entry points take, spread over their logarithm."""
    def over(lo, hi):
        return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi))))))
    while True:
        M, N, K = over(1, 20000), 8 * over(1, 2200), 8 * over(1, 2200)
        if M * N * K < 3e12:
            return product(op, M, N, K)


def check_cover(p, M, N, K):
    tm, tn = TILES[p.tile]
    tiles = -(-M // tm) * -(-N // tn)
    if p.tile != WIDE:
        if p.tile == FEW:
            assert M <= 16 and p.splits == 1 and p.bytes == 0
            return
        # parts of whole stages, none of them empty
        assert p.part % STAGE == 0 and p.part > 0
        assert (p.splits - 1) * p.part < K <= p.splits * p.part
        assert p.bytes == (p.splits * M * N * 4 if p.splits > 1 else 0)
        return
    assert p.whole + p.rest == tiles
    if not p.rest:
        assert p.whole == tiles and p.bytes == 0
        return
    # as the kernel places a piece: parts of `main` from 0 on, then what is left, in one piece or in `cuts` of `cut`
    left = p.rest - p.tails
    pieces = p.parts * p.rest + p.tails + left * p.cuts
    assert p.bytes == pieces * 256 * 256 * 4
    assert p.main % STAGE == 0 and p.main > 0 and p.cut % STAGE == 0 and 0 <= left < p.rest + 1
    at = p.parts * p.main
    assert (p.parts - 1) * p.main < K
    if not p.cut:
        assert p.tails == 0 and p.cuts == 0 and at >= K
        return
    assert at < K
    if left:
        assert p.cuts >= 1 and at + (p.cuts - 1) * p.cut < K <= at + p.cuts * p.cut


@pytest.mark.parametrize("op", [FWD, DGRAD, WGRAD])
def test_parts_cover_each_reduction_once(plan, op):
    rng = random.Random(op)
    for _ in range(20000):
        s = sizes(rng, op)
        check_cover(plan(op, *s), *s)


@pytest.mark.parametrize("op", [FWD, DGRAD, WGRAD])
@pytest.mark.parametrize("M,N,K", [(1 << 23, 8, 8), (1 << 23, 1 << 15, 8), (1 << 21, 1 << 17, 1 << 17), (17, 1 << 17, 1 << 17),
                                   (1, 8, 1 << 17), (1 << 23, 8, 1 << 15)])
def test_the_largest_sizes(plan, op, M, N, K):
    s = product(op, M, N, K)
    p = plan(op, *s)
    check_cover(p, *s)
    if op != WGRAD:
        assert ptm.pt_linear_workspace_size((ptm.PT_OP_FWD, ptm.PT_OP_DGRAD)[op], M, N, K) == p.bytes
    tm, tn = TILES[p.tile]
    # a launch stays below 2^32 threads
    assert -(-s[0] // tm) * -(-s[1] // tn) * p.splits * 256 < 1 << 32 or p.tile == FEW


def test_every_kind_is_compared_bit_for_bit(plan):
    """Also after a change of the planner's costs: a size that no longer takes its tile shows here."""
    have = set()
    for op in (FWD, DGRAD, WGRAD):
        for s in SHAPES:
            have.add((op,) + kind(plan(op, *product(op, *s))))
        for s in PRODUCTS + KINDS:
            have.add((op,) + kind(plan(op, *s)))
    for op, tiles in ((FWD, FWD_TILES + FORWARDS), (DGRAD, DGRAD_TILES), (WGRAD, WGRAD_TILES)):
        have.update((op,) + kind(plan(op, *product(op, *s))) for s in tiles)
    rng = random.Random(1)
    missing = {}
    for i in range(120000):
        op = i % 3
        s = sizes(rng, op)
        k = (op,) + kind(plan(op, *s))
        if k not in have:
            missing.setdefault(k, call(op, *s))
    assert not missing
