"""examples/moe_block.py with its shared expert and the norms behind it: the
joins of rows, the dense products and the block norm together with the router
and the experts, forward and backward, against autograd in 64 bits on the CPU.

Tolerances in the 2-norm, counted as in test_gpu_moe_block: a tensor stored in
bf16 is off by 2^-8 of its size at most.  The longest chains are
  out              y, c, h, o (or the shared expert's output), out          5
  after, y2        stream and the five above, after, y2                     8
  gradients        the first seven of those, then dout, do, dc, da, dy      15
                   (rounded once each for experts, router, shared), ds
"""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu

F64 = torch.float64
UNIT = 2.0 ** -8
NAMES = ("norm", "router", "w1", "w2", "s1", "s2", "post", "gate", "next")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(a, b):
    return (torch.linalg.norm(a.cpu().to(F64) - b) / torch.linalg.norm(b)).item()


def make(example, dev, T, H, I, E, k, S):
    block = example.MoeBlock(H, I, E, k, dev, seed=3, shared=S)
    g = torch.Generator(device=dev).manual_seed(4)
    for n in ("norm", "post", "gate", "next"):
        getattr(block, n).copy_(torch.rand(H, generator=g, device=dev) + 0.5)
    return block, [torch.randn((T, H), generator=g, device=dev).bfloat16() for _ in range(4)]


def normed(v, w):
    return v * (v.square().mean(1, keepdim=True) + 1e-5).pow(-0.5) * w


def glu(c):
    g, u = c.chunk(2, 1)
    return g * torch.sigmoid(g) * u


def reference(block, x, residual, ids):
    """The block and its close in 64 bits on the same choice of experts."""
    p = {n: getattr(block, n).cpu().to(F64).requires_grad_(True) for n in NAMES}
    stream = (x.cpu().to(F64) + residual.cpu().to(F64)).requires_grad_(True)
    y = normed(stream, p["norm"])
    w = torch.softmax((y @ p["router"].t()).gather(1, ids.cpu().long()), 1)
    out = glu(y @ p["s1"].t()) @ p["s2"].t()
    for e in range(block.E):
        t, j = torch.nonzero(ids.cpu() == e, as_tuple=True)
        out = out.index_add(0, t, glu(y[t] @ p["w1"][e].t()) @ p["w2"][e].t() * w[t, j].unsqueeze(1))
    after = stream + p["gate"] * normed(out, p["post"])
    return p, stream, out, after, normed(after, p["next"])


SHAPES = [(50, 128, 96, 8, 2, 64), (300, 256, 160, 12, 4, 192), (1, 64, 32, 8, 3, 32)]


@pytest.mark.parametrize("T,H,I,E,k,S", SHAPES)
def test_training_step(dev, example, T, H, I, E, k, S):
    block, (x, residual, dy2, dafter) = make(example, dev, T, H, I, E, k, S)
    out, stream = block.forward(x, residual)
    after, y2 = block.close(out, stream)
    ds = block.backward(*block.close_backward(dy2, dafter))
    torch.cuda.synchronize()
    p, s, rout, rafter, ry2 = reference(block, x, residual, block.saved[4])
    assert rel(out, rout) <= 5 * UNIT
    assert rel(after, rafter) <= 8 * UNIT
    assert rel(y2, ry2) <= 8 * UNIT
    ((ry2 * dy2.cpu().to(F64)).sum() + (rafter * dafter.cpu().to(F64)).sum()).backward()
    assert rel(ds, s.grad) <= 15 * UNIT
    for n in NAMES:
        assert rel(block.grad[n], p[n].grad) <= 15 * UNIT, n


@pytest.mark.parametrize("T,H,I,E,k,S", SHAPES)
def test_decode(dev, example, T, H, I, E, k, S):
    block, (x, residual, _, _) = make(example, dev, T, H, I, E, k, S)
    x, residual = x[:64], residual[:64]
    block.forward(x, residual)
    few, stream = block.decode(x, residual)
    assert torch.equal(stream, block.saved[0])
    assert rel(few, reference(block, x, residual, block.saved[4])[2]) <= 5 * UNIT


def test_a_captured_step(dev, example):
    """Replayed between eager steps of the same block and on other inputs: the eager step's bits, gradients included."""
    block, (x, residual, dy2, dafter) = make(example, dev, 300, 256, 160, 8, 2, 96)

    def step():
        for g in block.grad.values():
            g.zero_()
        after, y2 = block.close(*block.forward(x, residual))
        return [after, y2, block.backward(*block.close_backward(dy2, dafter))] + list(block.grad.values())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(4):
        g = torch.Generator(device=dev).manual_seed(seed)
        for t in (x, residual, dy2, dafter):
            t.copy_(torch.randn(t.shape, generator=g, device=dev))
        eager = [t.clone() for t in step()]
        for g in block.grad.values():
            g.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [[7], [0, 1, 49]])
def test_tokens_without_experts_and_memory_of_nan(dev, example, bad):
    """Rows that no expert has stay unwritten, and hold NaN here: no other token's output or gradient sees them."""
    T, H, I, E, k, S = 50, 128, 96, 8, 2, 64

    def of_nan(shape, dtype=torch.bfloat16):
        t = torch.empty(shape, dtype=dtype, device=dev)
        return t.fill_(float("nan")) if dtype.is_floating_point else t

    keep = [t for t in range(T) if t not in bad]
    alone, (x, residual, dout, dstream) = make(example, dev, T, H, I, E, k, S)
    ref, _ = alone.forward(x[keep], residual[keep])
    dref = alone.backward(dout[keep], dstream[keep])
    block, _ = make(example, dev, T, H, I, E, k, S)
    block._new = of_nan
    x[bad, 5] = float("nan")
    out, _ = block.forward(x, residual)
    ds = block.backward(dout, dstream)
    torch.cuda.synchronize()
    assert rel(out[keep], ref.cpu().to(F64)) <= 5 * UNIT
    assert rel(ds[keep], dref.cpu().to(F64)) <= 15 * UNIT
    for n in ("w1", "w2"):
        assert rel(block.grad[n], alone.grad[n].cpu().to(F64)) <= 15 * UNIT, n
