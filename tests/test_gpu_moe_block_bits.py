"""The bits that examples/moe_block.py keeps in its backward: the router's gradient
goes through its products as the fp32 values that it is, and the gradient at the
norm's output is rounded after the experts' sum and once more as a whole.

Tolerances, derived.  A reduction of K products in fp32 is off by (K / 16 + 64)
2^-23 of the sum of their sizes (test_gpu_linear); an fp32 value in three bf16
parts is exact, its parts' sizes at most 1 + 2^-7 of its own.  A rounding to bf16
is off by 2^-8 of the value.
"""
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm
from test_gpu_moe_block_whole import F64, UNIT, example, make  # noqa: F401

pytestmark = pytest.mark.gpu


def watch(monkeypatch, module, name, keep):
    real = getattr(module, name)

    def run(*args, **kw):
        real(*args, **kw)
        keep(args, kw)

    monkeypatch.setattr(module, name, run)


@pytest.mark.parametrize("T,H,I,E,k,S", [(50, 128, 96, 8, 2, 64), (300, 256, 160, 32, 4, 192), (300, 256, 160, 12, 4, 192),
                                         (257, 128, 64, 16, 3, 0), (1, 64, 32, 10, 3, 32)])
def test_the_routers_and_the_norms_gradients(dev, example, monkeypatch, T, H, I, E, k, S):  # noqa: F811
    block, (x, residual, dout, dstream) = make(example, dev, T, H, I, E, k, S)
    block.forward(x, residual)
    seen = {}
    watch(monkeypatch, ptm, "pt_moe_route_bwd", lambda a, kw: seen.update(dlogits=a[3].clone()))
    watch(monkeypatch, ptm, "pt_moe_combine", lambda a, kw: seen.update(da=a[0].clone(), row_of=a[2].clone()))
    watch(monkeypatch, ptm, "pt_rmsnorm_bwd", lambda a, kw: seen.update(dy=a[0].clone()))

    def shared(a, kw):
        if ptm.PT_ACT_SWIGLU in (kw.get("act"), *a[8:9]):
            seen["dsc"] = a[4].clone()

    watch(monkeypatch, ptm, "pt_linear_dgrad", shared)
    start = torch.randn(block.grad["router"].shape, device=dev)
    block.grad["router"].copy_(start)
    block.backward(dout, dstream)
    torch.cuda.synchronize()
    dl, y = seen["dlogits"].to(F64), block.saved[1].to(F64)
    assert seen["dlogits"].dtype == torch.float32
    want, size = dl.t() @ y, dl.abs().t() @ y.abs()
    off = (T / 16 + 64) * 2.0 ** -23 * 1.01 * size + 4 * 2.0 ** -24 * (size + start.to(F64).abs())
    assert ((block.grad["router"].to(F64) - want - start.to(F64)).abs() <= off).all()

    experts = seen["da"].to(F64)[seen["row_of"].long()].sum(1)
    terms = [(dl, block.router.to(F64))] + ([(seen["dsc"].to(F64), block.s1.to(F64))] if S else [])
    want = experts + sum(a @ w for a, w in terms)
    size = sum(a.abs() @ w.abs() for a, w in terms) + seen["da"].to(F64)[seen["row_of"].long()].abs().sum(1)
    off = UNIT * experts.abs() + ((2 * S + 3 * E) / 16 + 64 + k) * 2.0 ** -23 * 1.01 * size
    off = off + UNIT * (want.abs() + off)
    assert ((seen["dy"].to(F64) - want).abs() <= off).all()


def test_decoding_keeps_nothing_for_a_backward(dev, example, monkeypatch):  # noqa: F811
    """The same bits as the forward's shared expert, without its sums being stored."""
    T, H, I, E, k, S = 7, 128, 96, 8, 2, 64
    block, (x, residual, _, _) = make(example, dev, T, H, I, E, k, S)
    few, _ = block.decode(x, residual)
    kept = []
    watch(monkeypatch, ptm, "pt_linear_fwd", lambda a, kw: kept.append(a[5]))
    again, _ = block.decode(x, residual)
    torch.cuda.synchronize()
    assert torch.equal(few, again)
    assert len(kept) == 3 and all(c is None for c in kept)
    block.forward(x, residual)
    assert any(c is not None for c in kept[3:])
