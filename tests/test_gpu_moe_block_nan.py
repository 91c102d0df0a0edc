"""examples/moe_block.py with a token that holds a NaN: it has no experts, so
fewer rows than tokens times k are owned.  The other tokens' outputs and
gradients, and the experts', are those of a batch without it: the same rows in
the same order inside an expert, whose sums may be split at other places (the
tolerances of test_gpu_moe_block).
"""
import pytest
import torch

from test_gpu_moe_block import F64, example, rel  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [[7], [0, 1, 49]])
def test_a_token_with_a_nan(dev, example, bad):  # noqa: F811
    T, H, I, E, k = 50, 128, 96, 8, 2
    g = torch.Generator(device=dev).manual_seed(4)
    x, residual, dout, dstream = (torch.randn((T, H), generator=g, device=dev).bfloat16() for _ in range(4))
    keep = [t for t in range(T) if t not in bad]
    alone = example.MoeBlock(H, I, E, k, dev, seed=3)
    ref, _ = alone.forward(x[keep], residual[keep])
    dref = alone.backward(dout[keep], dstream[keep])

    block = example.MoeBlock(H, I, E, k, dev, seed=3)
    x[bad, 5] = float("nan")
    out, stream = block.forward(x, residual)
    ds = block.backward(dout, dstream)
    few, _ = block.decode(x, residual)
    torch.cuda.synchronize()
    assert stream[bad, 5].isnan().all()
    assert block.saved[4][bad].eq(-1).all() and block.saved[4][keep].ge(0).all()
    assert out[bad].eq(0).all() and few[bad].eq(0).all()
    assert rel(out[keep], ref.cpu().to(F64)) <= 4 * 2.0 ** -8
    assert rel(few[keep], ref.cpu().to(F64)) <= 4 * 2.0 ** -8
    assert rel(ds[keep], dref.cpu().to(F64)) <= 8 * 2.0 ** -8
    for n in ("w1", "w2"):
        assert rel(block.grad[n], alone.grad[n].cpu().to(F64)) <= 8 * 2.0 ** -8, n


def test_no_token_has_experts(dev, example):  # noqa: F811
    block = example.MoeBlock(128, 96, 8, 2, dev, seed=3)
    x = torch.full((20, 128), float("nan"), device=dev).bfloat16()
    out, _ = block.forward(x, torch.zeros_like(x))
    block.backward(torch.ones_like(x), torch.zeros_like(x))
    torch.cuda.synchronize()
    assert out.eq(0).all() and block.grad["w1"].eq(0).all() and block.grad["w2"].eq(0).all()
