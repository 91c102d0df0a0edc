"""The MoE router on the GPU against a plain implementation in 64 bits.

Choices, counts and orders are whole numbers and must be equal.  Weights
(fp32): exp, a sum of at most 1024 positive terms in a tree at most 22 deep,
a quotient and a product: 40 * 2^-24 of the value covers them (exp of an
argument up to 32 in size, itself rounded, adds 32 * 2^-24).  bf16 gradients
add a rounding of 2^-8.
"""
import numpy as np
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm

pytestmark = pytest.mark.gpu

F64 = torch.float64
LOGITS = {"f32": (ptm.PT_FP32, torch.float32), "bf16": (ptm.PT_BF16, torch.bfloat16)}
TOL = 80 * 2.0 ** -24
NINF = float("-inf")


def choose64(z, bias, k, gate, renorm, scale):
    """ids [T, k] (-1: none left) and weights in 64 bits, on the CPU."""
    z = z.detach().cpu().to(F64)
    z = torch.where(z.isnan(), torch.full_like(z, NINF), z)
    T, E = z.shape
    if gate == ptm.PT_GATE_SIGMOID:
        prob = 1 / (1 + torch.exp(-z))
        score = prob + (bias.cpu().to(F64) if bias is not None else 0)
        score = torch.where(z.isinf() & (z < 0), torch.full_like(z, NINF), score).float()   # fp32 scores, as documented
        score = torch.where(score.isnan(), torch.full_like(score, NINF), score)
    else:
        m = z.amax(1, keepdim=True)
        prob = torch.where(m > NINF, torch.exp(z - m), torch.zeros_like(z))
        prob = prob / prob.sum(1, keepdim=True).clamp(min=1e-300)
        score = z
    top, ids = torch.sort(score, dim=1, descending=True, stable=True)
    ok = top[:, :k] > NINF
    ids = ids[:, :k]
    w = torch.where(ok, prob.gather(1, ids), torch.zeros((), dtype=F64))
    if renorm:
        total = w.sum(1, keepdim=True)
        if gate == ptm.PT_GATE_SOFTMAX:          # a softmax over the chosen, however small next to the rest
            zc = torch.where(ok, z.gather(1, ids), torch.full_like(w, NINF))
            mc = zc.amax(1, keepdim=True)
            w = torch.where(ok, torch.exp(zc - mc), torch.zeros_like(w))
            total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return torch.where(ok, ids, torch.full_like(ids, -1)).int(), w * scale


def order64(ids, E):
    flat = ids.flatten().numpy()
    T, k = ids.shape
    lens = np.array([(flat == e).sum() for e in range(E)], np.int64)
    order = [i for e in np.argsort(np.where(flat < 0, E, flat), kind="stable").tolist() for i in [e]][: int(lens.sum())]
    row_of = np.full(T * k, -1, np.int32)
    row_of[order] = np.arange(len(order))
    token_of = np.full(T * k, -1, np.int32)
    token_of[: len(order)] = np.array(order, np.int64) // k
    return lens, row_of.reshape(T, k), token_of


def route(z, bias, k, gate, renorm, scale, ws="full"):
    T, E = z.shape
    dev = z.device
    dt = ptm.PT_BF16 if z.dtype == torch.bfloat16 else ptm.PT_FP32
    out = {"ids": torch.full((T, k), 99, dtype=torch.int32, device=dev), "w": torch.full((T, k), 7.0, device=dev),
           "lens": torch.full((E,), 99, dtype=torch.int64, device=dev),
           "row_of": torch.full((T, k), 99, dtype=torch.int32, device=dev),
           "token_of": torch.full((T * k,), 99, dtype=torch.int32, device=dev)}
    n = ptm.pt_moe_route_workspace_size(T, E, k)
    w = None if ws is None else torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=dev)
    if w is not None:
        w[:4] = 0
    ptm.pt_moe_route(z, bias, out["ids"], out["w"], out["lens"], out["row_of"], out["token_of"], T, E, k, dt, gate,
                     renorm, scale, workspace=None if w is None else w[:n])
    torch.cuda.synchronize()
    if w is not None:
        assert w[n:].eq(0xFF).all()
        out["err"] = ptm.pt_read_error_flags(w)
    return out


def check(z, bias, k, gate, renorm, scale, got):
    E = z.shape[1]
    ids, w = choose64(z, bias, k, gate, renorm, scale)
    assert torch.equal(got["ids"].cpu(), ids)
    assert ((got["w"].cpu().to(F64) - w).abs() <= TOL * w.abs() + 1e-37).all()
    lens, row_of, token_of = order64(ids, E)
    assert np.array_equal(got["lens"].cpu().numpy(), lens)
    assert np.array_equal(got["row_of"].cpu().numpy(), row_of)
    assert np.array_equal(got["token_of"].cpu().numpy(), token_of)


def logits(dev, T, E, seed, dtype="f32", shut=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    z = torch.randn((T, E), generator=g, device=dev) + 0.5 * torch.randn(E, generator=g, device=dev)
    if shut:
        z[:, torch.randperm(E, generator=g, device=dev)[:shut]] = NINF
    bias = 0.05 * torch.randn(E, generator=g, device=dev)
    return z.to(LOGITS[dtype][1]), bias


SIZES = [(1, 1, 1), (1, 8, 3), (3, 7, 7), (5, 256, 6), (63, 60, 4), (64, 32, 8), (65, 33, 2), (64, 1024, 16),
         (130, 17, 16), (200, 128, 8), (257, 512, 6), (1000, 257, 5), (70, 1001, 9), (4099, 32, 4)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("gate", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [0, 1])
def test_route(dev, T, E, k, gate, renorm):
    for dtype in ("f32", "bf16"):
        z, bias = logits(dev, T, E, T + E + k, dtype, shut=2 if E > k + 2 else 0)
        b = bias if gate else None
        got = route(z, b, k, gate, renorm, 2.5)
        assert got["err"] == 0
        check(z, b, k, gate, renorm, 2.5, got)


# up to 64 tokens whose choice is spread over workgroups, and parts of 16, of an odd number and of 64 tokens
@pytest.mark.parametrize("T,E,k", [(9, 1024, 16), (17, 256, 8), (33, 250, 5), (48, 100, 6), (64, 65, 12), (64, 257, 3), (300, 64, 4),
                                   (2500, 40, 4), (4101, 72, 6), (9000, 20, 2)])
@pytest.mark.parametrize("gate", [0, 1], ids=["softmax", "sigmoid"])
def test_choice_spread_over_workgroups(dev, T, E, k, gate):
    z, bias = logits(dev, T, E, T * 3 + E, "f32" if T % 2 else "bf16", shut=2)
    b = bias if gate else None
    got = route(z, b, k, gate, 1, 1.5)
    assert got["err"] == 0
    check(z, b, k, gate, 1, 1.5, got)
    z[T - 1, 3] = float("nan")
    z[T // 2] = NINF
    got = route(z, b, k, gate, 0, 1.5)
    assert got["err"] == 16
    check(z, b, k, gate, 0, 1.5, got)
    if T <= 64:
        bare = route(z, b, k, gate, 0, 1.5, ws=None)
        assert all(torch.equal(bare[n], got[n]) for n in bare)


def test_many_tokens_per_part(dev):
    # more than 256 chunks of 64 tokens: parts of several chunks
    z, _ = logits(dev, 40000, 24, 3, "bf16")
    check(z, None, 3, 0, 1, 1.0, route(z, None, 3, 0, 1, 1.0))


def test_no_tokens(dev):
    z = torch.empty((0, 16), device=dev)
    got = route(z, None, 2, 0, 1, 1.0)
    assert got["lens"].eq(0).all()


@pytest.mark.parametrize("gate", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [20, 90])
def test_ties_go_to_the_lower_index(dev, gate, T):
    z = torch.zeros((T, 100), device=dev)
    z[1] = -0.0
    z[2, 50:] = 1.0
    z[3, ::2] = -0.0                                     # signed zeros are equal
    z[4, 99] = 2.0
    z[5] = torch.arange(100, device=dev) % 3
    check(z, None, 6, gate, 1, 1.0, route(z, None, 6, gate, 1, 1.0))
    check(z.bfloat16(), None, 6, gate, 0, 1.0, route(z.bfloat16(), None, 6, gate, 0, 1.0))


@pytest.mark.parametrize("gate", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("T", [12, 100])
def test_rows_with_little_or_nothing_left(dev, gate, renorm, T):
    z, bias = logits(dev, T, 40, 8)
    z[0] = NINF                                          # nothing
    z[1] = NINF
    z[1, 7] = -3.0                                       # one
    z[2] = NINF
    z[2, 30:33] = torch.tensor([1.0, 1.0, 2.0], device=dev)
    z[3] = -3.4028234663852886e38                        # a mask of the type's lowest value is a number: all tie
    z[4] = -3.4028234663852886e38
    z[4, 11] = 0.0
    z[5] = -200.0                                        # fp32 sigmoids would all vanish
    z[6] = 90.0
    z[7] = 1e4
    b = bias if gate else None
    got = route(z, b, 5, gate, renorm, 1.0)
    assert got["err"] == 0
    check(z, b, 5, gate, renorm, 1.0, got)
    assert got["ids"][0].eq(-1).all() and got["w"][0].eq(0).all()
    assert got["w"].isfinite().all()


@pytest.mark.parametrize("gate", [0, 1], ids=["softmax", "sigmoid"])
def test_nan_is_never_chosen_and_is_reported(dev, gate):
    for T in (10, 100):
        z, _ = logits(dev, T, 64, 4)
        z[2, 5] = float("nan")
        z[3] = float("nan")
        got = route(z, None, 4, gate, 0, 1.0)
        check(z, None, 4, gate, 0, 1.0, got)
        assert got["err"] == 16 and got["ids"][3].eq(-1).all()


@pytest.mark.parametrize("T", [10, 100])
def test_infinite_biases(dev, T):
    z, bias = logits(dev, T, 64, 15)
    bias[5] = NINF
    check(z, bias, 4, 1, 1, 1.0, route(z, bias, 4, 1, 1, 1.0))
    bias[[9, 40]] = float("inf")                         # fewer than are chosen, then more
    check(z, bias, 4, 1, 0, 1.0, route(z, bias, 4, 1, 0, 1.0))
    bias[50:60] = float("inf")
    check(z, bias, 4, 1, 1, 1.0, route(z, bias, 4, 1, 1, 1.0))


def test_logits_past_32_bits(dev):
    """More than 2^31 logits: the last tokens' choices and gradients, and the counts."""
    T, E, k = 2_100_000, 1024, 2
    z = torch.zeros((T, E), dtype=torch.bfloat16, device=dev)
    tail, _ = logits(dev, 500, E, 16, "bf16")
    z[-500:] = tail
    n = ptm.pt_moe_route_workspace_size(T, E, k)
    ids, w = torch.empty((T, k), dtype=torch.int32, device=dev), torch.empty((T, k), device=dev)
    lens, row_of = torch.empty(E, dtype=torch.int64, device=dev), torch.empty((T, k), dtype=torch.int32, device=dev)
    token_of = torch.empty(T * k, dtype=torch.int32, device=dev)
    ptm.pt_moe_route(z, None, ids, w, lens, row_of, token_of, T, E, k, ptm.PT_BF16, 0, 1, 1.0,
                     workspace=torch.zeros(n, dtype=torch.uint8, device=dev))
    rids, rw = choose64(tail, None, k, 0, 1, 1.0)
    assert torch.equal(ids[-500:].cpu(), rids) and ((w[-500:].cpu().to(F64) - rw).abs() <= TOL * rw).all()
    assert ids[:-500].eq(torch.tensor([0, 1], device=dev, dtype=torch.int32)).all()
    flat = ids.flatten().long()
    assert torch.equal(lens, torch.bincount(flat, minlength=E))
    order = torch.argsort(flat, stable=True)
    assert torch.equal(token_of.long(), order // k)
    assert torch.equal(row_of.flatten()[order].long(), torch.arange(T * k, device=dev))
    dw = torch.ones((T, k), device=dev)
    dw[:, 1] = -1.0
    dz = torch.empty_like(z)
    ptm.pt_moe_route_bwd(z, ids, dw, dz, T, E, k, ptm.PT_BF16, 0, 1, 1.0)
    alone = backward(tail, ids[-500:].contiguous(), dw[-500:].contiguous(), 0, 1, 1.0)
    assert torch.equal(dz[-500:], alone)


@pytest.mark.parametrize("T", [10, 100])
def test_plus_infinity_is_chosen_first(dev, T):
    z, _ = logits(dev, T, 64, 14)
    z[1, 7] = float("inf")
    big = z.clone()
    big[1, 7] = 1e30
    for gate, renorm in ((0, 0), (0, 1), (1, 0), (1, 1)):
        got, ref = route(z, None, 4, gate, renorm, 1.0), route(big, None, 4, gate, renorm, 1.0)
        assert got["err"] == 0 and got["ids"][1, 0] == 7
        assert all(torch.equal(got[n], ref[n]) for n in ("ids", "lens", "row_of", "token_of"))
        keep = torch.arange(T, device=dev) != 1
        assert torch.equal(got["w"][keep], ref["w"][keep])
        # a softmax with +inf has no value; a sigmoid is 1 there
        assert got["w"][1].isnan().all() if gate == 0 else torch.equal(got["w"][1], ref["w"][1])


def test_scores_that_differ_in_their_last_bit(dev):
    """Sigmoid scores with a bias: the order is that of the fp32-rounded 64-bit scores, near 1 too."""
    g = torch.Generator(device=dev).manual_seed(2)
    z = 8 + 4 * torch.rand((300, 128), generator=g, device=dev)
    bias = 1e-3 * torch.randn(128, generator=g, device=dev)
    check(z, bias, 8, 1, 1, 1.0, route(z, bias, 8, 1, 1, 1.0))
    check(z, None, 8, 1, 0, 1.0, route(z, None, 8, 1, 0, 1.0))


def test_without_workspace_and_repeated(dev):
    z, _ = logits(dev, 64, 48, 6)
    a, b = route(z, None, 4, 0, 1, 1.0, ws=None), route(z, None, 4, 0, 1, 1.0)
    assert all(torch.equal(a[n], b[n]) for n in a)
    z, _ = logits(dev, 5000, 48, 6)
    a, b = route(z, None, 4, 0, 1, 1.0), route(z, None, 4, 0, 1, 1.0)
    assert all(torch.equal(a[n], b[n]) for n in a if n != "err")


# ------------------------------------------------------------------ backward
def weights64(z, ids, gate, renorm, scale):
    """The weights of fixed choices, in 64 bits and differentiable."""
    ok = ids >= 0
    at = ids.clamp(min=0).long()
    if gate == ptm.PT_GATE_SIGMOID:
        v = torch.sigmoid(z).gather(1, at)
        v = torch.where(ok, v, torch.zeros_like(v))
        if renorm:
            v = v / v.sum(1, keepdim=True).clamp(min=1e-300)
    elif renorm:
        zc = torch.where(ok, z.gather(1, at), torch.full_like(z[:, : ids.shape[1]], -1e30))
        v = torch.where(ok, torch.softmax(zc, 1), torch.zeros_like(zc))
    else:
        v = torch.where(ok, torch.softmax(z, 1).gather(1, at), torch.zeros((), dtype=F64))
    return v * scale


def backward(z, ids, dw, gate, renorm, scale):
    dt = ptm.PT_BF16 if z.dtype == torch.bfloat16 else ptm.PT_FP32
    dz = torch.full_like(z, 7.0)
    ptm.pt_moe_route_bwd(z, ids, dw, dz, z.shape[0], z.shape[1], ids.shape[1], dt, gate, renorm, scale)
    torch.cuda.synchronize()
    return dz


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("gate", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [0, 1])
def test_backward(dev, T, E, k, gate, renorm):
    for dtype in ("f32", "bf16"):
        z, _ = logits(dev, T, E, T * 3 + E, dtype, shut=2 if E > k + 2 else 0)
        ids = route(z, None, k, gate, renorm, 2.5)["ids"]
        dw = torch.randn((T, k), generator=torch.Generator(device=dev).manual_seed(5), device=dev)
        dz = backward(z, ids, dw, gate, renorm, 2.5)
        z64 = z.cpu().to(F64).requires_grad_(True)
        w = weights64(z64, ids.cpu(), gate, renorm, 2.5)
        (w * dw.cpu().to(F64)).sum().backward()
        ref = torch.where(z64.isinf(), torch.zeros_like(z64), z64.grad).nan_to_num(0.0)
        # a sum of k terms of both signs times the share: rounding errors go by the largest term
        big = 2.5 * dw.cpu().to(F64).abs().amax(1, keepdim=True)
        half = torch.finfo(z.dtype).eps / 2
        assert ((dz.cpu().to(F64) - ref).abs() <= half * ref.abs() + TOL * big * (1 if gate == 0 else 1)).all()
        assert dz[z.isinf()].eq(0).all()


@pytest.mark.parametrize("gate", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [0, 1])
def test_backward_edges_and_differences(dev, gate, renorm):
    z, _ = logits(dev, 9, 40, 8)
    z[0] = NINF
    z[1] = NINF
    z[1, 7] = -3.0
    z[2] = 30.0 + z[2] / 8                               # sigmoids that round to 1
    z[3] = -200.0
    ids = route(z, None, 5, gate, renorm, 1.5)["ids"]
    ids[4, 2] = -1                                       # a slot without an expert
    ids[5, 0] = 1 << 20                                  # and one outside every table
    dw = torch.randn((9, 5), generator=torch.Generator(device=dev).manual_seed(5), device=dev)
    dz = backward(z, ids, dw, gate, renorm, 1.5)
    assert dz.isfinite().all() and dz[0].eq(0).all()
    use = torch.where(ids >= 40, torch.full_like(ids, -1), ids).cpu()
    z64 = torch.where(z.isinf(), torch.full_like(z, -1e4), z).cpu().to(F64)
    dirn = torch.randn((9, 40), generator=torch.Generator().manual_seed(6), dtype=F64)
    dirn[z.cpu().isinf()] = 0

    def loss(t):
        return (weights64(z64 + t * dirn, use, gate, renorm, 1.5) * dw.cpu().to(F64))[1:].sum().item()

    t = 1e-5
    numeric = (loss(t) - loss(-t)) / (2 * t)
    ours = (dz.cpu().to(F64) * dirn)[1:].sum().item()
    slack = TOL * (1.5 * dw.abs().amax().item()) * dirn.abs().sum().item() + 1e-7
    assert abs(numeric - ours) <= slack
    if gate == 1 and renorm == 0:                        # v (1 - v) keeps its digits where v rounds to 1
        v = torch.sigmoid(-z[2].cpu().to(F64))
        at = ids[2].cpu().long()
        want = (v * (1 - v))[at] * dw[2].cpu().to(F64) * 1.5
        assert ((dz[2].cpu().to(F64)[at] - want).abs() <= TOL * want.abs()).all()


def test_graph_replays(dev):
    z, bias = logits(dev, 700, 60, 12)
    eager = route(z, bias, 4, 1, 1, 1.0)
    out = {n: torch.zeros_like(t) for n, t in eager.items() if n != "err"}
    dw = torch.ones((700, 4), device=dev)
    ref = backward(z, eager["ids"], dw, 1, 1, 1.0)
    dz = torch.zeros_like(z)
    ws = torch.zeros(ptm.pt_moe_route_workspace_size(700, 60, 4), dtype=torch.uint8, device=dev)

    def run():
        ptm.pt_moe_route(z, bias, out["ids"], out["w"], out["lens"], out["row_of"], out["token_of"], 700, 60, 4,
                         ptm.PT_FP32, 1, 1, 1.0, workspace=ws)
        ptm.pt_moe_route_bwd(z, out["ids"], dw, dz, 700, 60, 4, ptm.PT_FP32, 1, 1, 1.0)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for t in (*out.values(), dz, ws):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], eager[n]) for n in out) and torch.equal(dz, ref)
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], eager[n]) for n in out) and torch.equal(dz, ref)
