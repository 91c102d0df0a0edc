"""Sigmoid routing with a bias of fp32's lowest value, the usual mask of an
expert: a number like any other, so masked experts follow the open ones, the
lower index first, while an expert whose logit is -inf is never chosen.  Against
the plain implementation in 64 bits of test_gpu_route, with its tolerances.
"""
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm
from test_gpu_few_tokens import KINDS, check as check_layer, make
from test_gpu_route import NINF, check, logits, route

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min


def masked(bias, E, mask):
    """Three open experts, one shut by its logit with an ordinary bias, the others masked."""
    shut = E // 2
    b = torch.full_like(bias, mask)
    keep = [1, E // 3, E - 1, shut]
    b[keep] = bias[keep]
    return b, shut


# experts that fill their lanes and that do not; one workgroup, a choice by several, parts of tokens
@pytest.mark.parametrize("E", [8, 24, 32, 40, 60, 64, 100, 128, 250, 256, 500, 1000, 1024])
@pytest.mark.parametrize("T", [1, 5, 30, 64, 300])
@pytest.mark.parametrize("mask", [LOWEST, LOWEST * (1 - 2.0 ** -21)])
def test_lowest_bias(dev, T, E, mask):
    z, bias = logits(dev, T, E, T + E)
    b, shut = masked(bias, E, mask)
    z[:, shut] = NINF
    for k in (2, 3, 6):                                  # fewer than are open, all of them, and more
        for dtype in (torch.float32, torch.bfloat16):
            got = route(z.to(dtype), b, k, ptm.PT_GATE_SIGMOID, 1, 2.5)
            assert got["err"] == 0
            check(z.to(dtype), b, k, ptm.PT_GATE_SIGMOID, 1, 2.5, got)
            assert got["ids"].ne(shut).all() and got["ids"].lt(E).all() and got["ids"].ge(0).all()


def test_lowest_bias_next_to_infinities_and_nan(dev):
    for T, E in ((5, 60), (40, 256), (300, 40)):
        z, bias = logits(dev, T, E, 7)
        b, shut = masked(bias, E, LOWEST)
        z[:, shut] = NINF
        b[0] = NINF                                      # never, whatever its logit
        b[2] = float("inf")                              # always first
        z[T // 2] = NINF
        z[T - 1, 3:] = NINF                              # three left, one of them masked for good
        check(z, b, 6, ptm.PT_GATE_SIGMOID, 0, 1.0, route(z, b, 6, ptm.PT_GATE_SIGMOID, 0, 1.0))
        z[0, 4] = float("nan")
        got = route(z, b, 6, ptm.PT_GATE_SIGMOID, 0, 1.0)
        assert got["err"] == 16
        check(z, b, 6, ptm.PT_GATE_SIGMOID, 0, 1.0, got)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("T,E", [(1, 60), (9, 40), (40, 256)])
def test_lowest_bias_in_the_few_token_layer(dev, T, E, kind):
    x, z, bias, ops = make(dev, T, E, 96, 64, kind, T + E)
    b, shut = masked(bias, E, LOWEST)
    z[:, shut] = NINF
    check_layer(x, z, b, ops, 6, ptm.PT_GATE_SIGMOID, 1, 2.5, kind)
