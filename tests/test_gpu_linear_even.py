"""The widest tile with the reduction of its last tiles cut so that all compute
units end together: in equal parts, in parts and tails, with tails in pieces, with
and without whole tiles before.  Integer operands, bit for bit against exact sums
(below 2^24), whole and with what each epilogue does."""
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm
from test_gpu_linear import BF16, F32, dgrad, forward, gen, ints, wgrad

pytestmark = pytest.mark.gpu

# rows, columns and reduction of the product that is computed
PRODUCTS = [(8200, 392, 6152), (520, 10256, 8200), (4104, 2064, 5128), (392, 5136, 16392), (1040, 16400, 2056), (12296, 136, 8200),
            (16392, 144, 5128), (8200, 144, 16392), (3080, 5136, 1032), (16392, 1040, 3080), (1032, 5136, 10248)]


def test_the_products_are_cut():
    for M, N, K in PRODUCTS:
        assert ptm.pt_linear_workspace_size(ptm.PT_OP_FWD, M, N, K) and ptm.pt_linear_workspace_size(ptm.PT_OP_DGRAD, M, K, N)
        assert ptm.pt_linear_workspace_size(ptm.PT_OP_WGRAD, K, M, N)


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_forward(dev, M, N, K):
    g = gen(dev, M + N + K)
    x, w, bias, res = ints(g, M, K, top=1), ints(g, N, K, top=1), ints(g, N, top=20), ints(g, M, N, top=50)
    c = x.float() @ w.float().t() + bias.float()
    out, saved = forward(x, w, bias, res.float(), out_type=F32, save=True)
    assert torch.equal(out, c + res.float()) and torch.equal(saved, c.to(BF16))
    own = res.clone()
    assert torch.equal(forward(x, w, bias, own, out=own), (c + res.float()).to(BF16))
    if N % 16:
        return
    I = N // 2
    w[:I] = 0
    bias[:I] = (128 + torch.arange(I, device=dev) % 64).to(BF16)          # silu is the identity
    up = c[:, I:]
    out, saved = forward(x, w, bias, act="swiglu", out_type=F32, save=True)
    assert torch.equal(out, bias[:I].float() * up) and torch.equal(saved[:, I:], up.to(BF16))
    assert torch.equal(saved[:, :I], bias[:I].expand(M, I))


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_dgrad(dev, M, N, K):
    g = gen(dev, M + N + K + 1)
    dy, w, add = ints(g, M, K, top=1), ints(g, K, N, top=1), ints(g, M, N, top=50)
    dh = dy.float() @ w.float()
    own = add.clone()
    assert torch.equal(dgrad(dy, w, add=own, dx=own), (dh + add.float()).to(BF16))
    c = torch.empty((M, 2 * N), dtype=BF16, device=dev)
    c[:, :N] = (128 + torch.arange(N, device=dev) % 64).to(BF16)
    c[:, N:] = ints(g, M, N)
    got = dgrad(dy, w, c, act="swiglu")
    assert torch.equal(got[:, :N], (dh * c[:, N:].float()).to(BF16))
    assert torch.equal(got[:, N:], (dh * c[:, :N].float()).to(BF16))


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_wgrad(dev, M, N, K):
    g = gen(dev, M + N + K + 2)
    dy, x = ints(g, K, M, top=1), ints(g, K, N, top=1)
    dw, db = dy.float().t() @ x.float(), dy.float().sum(0)
    got, gotb = wgrad(x, dy)
    assert torch.equal(got, dw) and torch.equal(gotb, db)
    start, startb = ints(g, M, N, top=50).float(), ints(g, M, top=50).float()
    got, gotb = wgrad(x, dy, accumulate=1, main_grad=start.clone(), dbias=startb.clone())
    assert torch.equal(got, dw + start) and torch.equal(gotb, db + startb)
    again, _ = wgrad(x, dy)
    assert torch.equal(again, dw)
