"""The router's gradient, element by element against 64 bits, each within the
roundings of its own terms: 80 * 2^-24 of them (the exponentials' arguments, the
sum and the quotient of test_gpu_route) and half a step of the output's type.

With g = scale dweights, p the softmax, v the sigmoids and w the weights of the
chosen ones without the scale, the terms of expert e are
    softmax           p_e (|g_e| + sum_j p_j |g_j|),   g_e = 0 where not chosen
    softmax, renorm   w_e (|g_e| + sum_j w_j |g_j|)    over the chosen
    sigmoid           v (1 - v) |g|
    sigmoid, renorm   w_e (1 - v_e) (|g_e| + sum_j w_j |g_j|)
"""
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm
from test_gpu_route import F64, TOL, backward, logits, route

pytestmark = pytest.mark.gpu


def terms64(z, ids, g, gate, renorm):
    """The gradient and the sizes of its terms, in 64 bits on the CPU."""
    at = ids.long()
    if gate == ptm.PT_GATE_SOFTMAX and not renorm:
        p = torch.softmax(z, 1)
        full = torch.zeros_like(z).scatter_(1, at, g)
        return p * (full - (p * full).sum(1, keepdim=True)), p * (full.abs() + (p * full.abs()).sum(1, keepdim=True))
    zc = z.gather(1, at)
    v = torch.sigmoid(zc)
    if gate == ptm.PT_GATE_SOFTMAX:
        w, tail = torch.softmax(zc, 1), 1.0
    elif renorm:
        w, tail = v / v.sum(1, keepdim=True), torch.sigmoid(-zc)
    if renorm:
        d = w * tail * (g - (w * g).sum(1, keepdim=True))
        big = w * tail * (g.abs() + (w * g.abs()).sum(1, keepdim=True))
    else:
        d = v * torch.sigmoid(-zc) * g
        big = d.abs()
    zero = torch.zeros_like(z)
    return zero.scatter(1, at, d), zero.scatter(1, at, big)


@pytest.mark.parametrize("T,E,k", [(1, 8, 3), (5, 256, 6), (300, 17, 16), (200, 60, 4), (200, 128, 8), (90, 256, 6), (60, 512, 6), (70, 1001, 9),
                                   (64, 1024, 16)])
@pytest.mark.parametrize("gate", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_each_element(dev, T, E, k, gate, renorm, dtype):
    z, _ = logits(dev, T, E, T * 5 + E, dtype)
    ids = route(z, None, k, gate, renorm, 2.5)["ids"]
    dw = torch.randn((T, k), generator=torch.Generator(device=dev).manual_seed(6), device=dev)
    dz = backward(z, ids, dw, gate, renorm, 2.5).cpu().to(F64)
    ref, big = terms64(z.cpu().to(F64), ids.cpu(), 2.5 * dw.cpu().to(F64), gate, renorm)
    half = torch.finfo(z.dtype).eps / 2
    assert ((dz - ref).abs() <= half * ref.abs() + TOL * (1 + half) * big).all()
