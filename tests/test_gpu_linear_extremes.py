"""Activations and their slopes at the ends of their range, on the GPU: every
activation's slope at large sums, and infinite sums.

An activation is taken in fp32 within 16 roundings of its terms, a slope likewise
and rounded to bf16 (2^-8).  At the values here sigmoids, tanh and erf are 0 or 1
or differ from them by less than the 1e-30 that is allowed beside that.
"""
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm
from test_gpu_linear import ACTS, BF16, F32, F64, act64, forward

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("act", [a for a in ACTS if a != "none"])
def test_slopes_of_large_sums(dev, act):
    vals = [120.0, -120.0, 300.0, -300.0, 1e4, -1e4, 1e18, -1e18]
    c = torch.tensor([vals], device=dev).to(BF16)
    if act == "swiglu":
        c = torch.cat([c, torch.full_like(c, 0.5)], 1)
    dc = torch.empty_like(c)
    ptm.pt_linear_act_bwd(torch.ones((1, 8), dtype=BF16, device=dev), c, dc, 1, c.shape[1], ACTS[act])
    c64 = c.to(F64).requires_grad_(True)
    want = torch.autograd.grad(act64(c64, act).sum(), c64)[0]
    assert torch.isfinite(want).all()
    assert ((dc.to(F64) - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs() + 1e-30).all()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M", [7, 100])
def test_infinite_sums(dev, act, M):
    """What the formula gives, an infinity or a NaN or 0; a slope is its limit or a NaN."""
    I = 8
    N = 2 * I if act == "swiglu" else I
    x, w, bias = torch.zeros((M, 8), dtype=BF16, device=dev), torch.zeros((N, 8), dtype=BF16, device=dev), torch.zeros(N, device=dev)
    bias[:I] = torch.tensor([INF, -INF, 1.0, -1.0, INF, -INF, 0.0, 2.0], device=dev)
    if act == "swiglu":
        bias[I:] = torch.tensor([0.5, 0.5, INF, -INF, -0.25, 2.0, 3.0, INF], device=dev)
    bias = bias.to(BF16)
    out, saved = forward(x, w, bias, out_type=F32, act=act, save=True)
    assert torch.equal(saved, bias.expand(M, N))
    want = act64(bias.to(F64).expand(M, N), act)
    torch.testing.assert_close(out.to(F64), want, rtol=2.0 ** -20, atol=1e-30, equal_nan=True)
    if act == "none":
        return
    if act == "swiglu":
        # the clamp makes +inf a number again
        out = forward(x, w, bias, out_type=F32, act=act, limit=3.0)
        want = act64(bias.to(F64).expand(M, N), act, 3.0)
        torch.testing.assert_close(out.to(F64), want, rtol=2.0 ** -20, atol=1e-30, equal_nan=True)
        return
    dc = torch.empty_like(saved)
    ptm.pt_linear_act_bwd(torch.ones((M, I), dtype=BF16, device=dev), saved, dc, M, N, ACTS[act])
    up, down = dc[:, [0, 4]], dc[:, [1, 5]]
    assert (torch.isnan(up) | (up == (INF if act == "relu2" else 1.0))).all()
    assert (torch.isnan(down) | (down == 0)).all()
    assert torch.isfinite(dc[:, [2, 3, 6, 7]]).all()
