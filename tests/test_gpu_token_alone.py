"""A token's bits do not depend on who shares its call: its row of a call over
many tokens equals a call of its own, bit for bit, whatever kernels, workgroups
and lanes the two calls are given.
"""
import pytest
import torch

from test_gpu_few_tokens import KINDS, make, run
from test_gpu_route import logits, route

pytestmark = pytest.mark.gpu


def weights(g, E, rows, cols, kind):
    """Operand and scales of E matrices, made on the GPU alone."""
    dev = g.device
    if kind == "bf16":
        return (torch.randn((E, rows, cols), generator=g, device=dev) * cols ** -0.5).bfloat16(), None
    s = torch.randint(117, 121, (E, rows, cols // 32), generator=g, device=dev).to(torch.uint8)
    if kind == "mxfp8":
        q = torch.randn((E, rows, cols), generator=g, device=dev).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        q = torch.randint(0, 256, (E, rows, cols // 2), generator=g, device=dev, dtype=torch.int32).to(torch.uint8)
    return q, s


# weight rows a multiple of 4096 bytes apart, whose tiles start at different places of them; 2 of 4 experts: one token
# runs in workgroups of 4 waves, 12 of 8 (of 16 where rows are 8192 values long) and 40 of 16
@pytest.mark.parametrize("kind,H,I", [("bf16", 4096, 2048), ("bf16", 2048, 4096), ("mxfp8", 4096, 4096), ("mxfp4", 8192, 8192)])
@pytest.mark.parametrize("T", [12, 40])
def test_rows_whose_tiles_take_turns(dev, T, kind, H, I):
    g = torch.Generator(device=dev).manual_seed(T + H)
    w1, s1 = weights(g, 4, 2 * I, H, kind)
    w2, s2 = weights(g, 4, H, I, kind)
    x = torch.randn((T, H), generator=g, device=dev).bfloat16()
    z = torch.randn((T, 4), generator=g, device=dev)
    many, _, _ = run(x, z, None, w1, s1, w2, s2, 2, 0, 1, 1.0, kind)
    alone = torch.cat([run(x[t:t + 1].clone(), z[t:t + 1].clone(), None, w1, s1, w2, s2, 2, 0, 1, 1.0, kind)[0]
                       for t in range(T)])
    assert many.float().isfinite().all() and torch.equal(alone, many)


@pytest.mark.parametrize("E,k", [(20, 8), (30, 10), (60, 4), (64, 9), (100, 5), (128, 6), (256, 6), (250, 16), (512, 6), (1024, 4)])
@pytest.mark.parametrize("gate", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [0, 1])
def test_router(dev, E, k, gate, renorm):
    """The choice and the weights, with as many lanes and experts to a lane as each number of tokens gets."""
    z, bias = logits(dev, 300, E, E + k)
    b = bias if gate else None
    many = route(z, b, k, gate, renorm, 2.5)
    for T in (1, 12, 20, 40, 64, 130):
        few = route(z[:T].clone(), b, k, gate, renorm, 2.5)
        assert torch.equal(few["ids"], many["ids"][:T]) and torch.equal(few["w"], many["w"][:T]), T


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_layer_with_shares_of_all_experts(dev, kind):
    x, z, _, (a, b) = make(dev, 40, 128, 96, 64, kind, 43)
    many, _, w = run(x, z, None, a[0], a[1], b[0], b[1], 6, 0, 0, 1.0, kind)
    for T in (1, 20):
        few, _, v = run(x[:T].clone(), z[:T].clone(), None, a[0], a[1], b[0], b[1], 6, 0, 0, 1.0, kind)
        assert torch.equal(v, w[:T]) and torch.equal(few, many[:T])
