"""The norm, the router, the grouped GEMMs and the few-token layer together, as
examples/moe_block.py uses them, against autograd in 64 bits on the CPU.

Tolerances in the 2-norm.  Every tensor that the block stores in bf16 is off by
2^-8 of its size at most, and independently; the longest chain of them on the way
to an output is y, c or h, o, out (forward: 4), and dout's row, dc, da, dy, ds
behind y, c, h (backward: 8).  Sums of that many independent errors in
quadrature stay below 2^-8 times their number: 4 * 2^-8 and 8 * 2^-8.
"""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(a, b):
    return (torch.linalg.norm(a.cpu().to(F64) - b) / torch.linalg.norm(b)).item()


def reference(block, x, residual, ids):
    """The block in 64 bits on the same choice of experts."""
    p = {n: getattr(block, n).cpu().to(F64).requires_grad_(True) for n in ("norm", "router", "w1", "w2")}
    stream = (x.cpu().to(F64) + residual.cpu().to(F64)).requires_grad_(True)
    y = stream * (stream.square().mean(1, keepdim=True) + 1e-5).pow(-0.5) * p["norm"]
    z = y @ p["router"].t()
    w = torch.softmax(z.gather(1, ids.cpu().long()), 1)
    out = torch.zeros_like(stream)
    for e in range(block.E):
        t, j = torch.nonzero(ids.cpu() == e, as_tuple=True)
        c = y[t] @ p["w1"][e].t()
        g, u = c.chunk(2, 1)
        out = out.index_add(0, t, (g * torch.sigmoid(g) * u) @ p["w2"][e].t() * w[t, j].unsqueeze(1))
    return p, stream, out


@pytest.mark.parametrize("T,H,I,E,k", [(50, 128, 96, 8, 2), (300, 256, 160, 12, 4)])
def test_training_step(dev, example, T, H, I, E, k):
    block = example.MoeBlock(H, I, E, k, dev, seed=3)
    g = torch.Generator(device=dev).manual_seed(4)
    x, residual, dout, dstream = (torch.randn((T, H), generator=g, device=dev).bfloat16() for _ in range(4))
    out, stream = block.forward(x, residual)
    ds = block.backward(dout, dstream)
    torch.cuda.synchronize()
    p, s, ref = reference(block, x, residual, block.saved[4])
    assert rel(out, ref) <= 4 * 2.0 ** -8
    (ref * dout.cpu().to(F64)).sum().backward()
    assert rel(ds, s.grad + dstream.cpu().to(F64)) <= 8 * 2.0 ** -8
    for n in ("norm", "router", "w1", "w2"):
        assert rel(block.grad[n], p[n].grad) <= 8 * 2.0 ** -8, n


def test_decode_agrees_with_the_forward(dev, example):
    block = example.MoeBlock(256, 160, 12, 4, dev, seed=5)
    g = torch.Generator(device=dev).manual_seed(6)
    x, residual = (torch.randn((64, 256), generator=g, device=dev).bfloat16() for _ in range(2))
    out, stream = block.forward(x, residual)
    few, stream2 = block.decode(x, residual)
    _, _, ref = reference(block, x, residual, block.saved[4])
    assert torch.equal(stream, stream2)
    assert rel(few, ref) <= 4 * 2.0 ** -8
    assert rel(few, out.cpu().to(F64)) <= 4 * 2.0 ** -8
