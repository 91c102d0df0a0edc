"""The whole MoE layer for a few tokens on the GPU against 64 bits.

Tolerance, derived: products are exact in fp32, sums have at most 16384 terms
in 8 chains of 64 lanes' MFMA order (512 * 2^-24 of the sum of the terms'
sizes covers them); h is rounded to bf16 (2^-8 of each h) and the output once
more (2^-8).  So, with S = sum over slots of w * sum_j |h_j w2_nj|,
    |out - ref| <= 2^-8 |ref| + (2^-8 + 2^-12) S + the FC1 sums' share,
the reference without the rounding of h; and in the 2-norm, where roundings
do not conspire, 2^-7 of the reference.  The FC1 sums: 512 * 2^-24 of
sum |x w1| in gate and up, taken through SwiGLU's slopes (at most 1.1 |up| and
|gate|).
"""
import numpy as np
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm
from test_gpu_route import choose64

pytestmark = pytest.mark.gpu

F64 = torch.float64
KINDS = {"bf16": ptm.PT_BF16, "mxfp8": ptm.PT_MXFP8_E4M3, "mxfp4": ptm.PT_MXFP4_E2M1}
GRID = [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]
NINF = float("-inf")


def weights(g, E, rows, cols, kind):
    """(operand, scales, values in 64 bits on the CPU) of E matrices with entries of about cols^-1/2."""
    dev = g.device
    if kind == "bf16":
        w = (torch.randn((E, rows, cols), generator=g, device=dev) * cols ** -0.5).bfloat16()
        return w, None, w.cpu().to(F64)
    e = int(np.floor(np.log2(cols ** -0.5)))
    s = torch.randint(127 + e - 2, 127 + e + 1, (E, rows, cols // 32), generator=g, device=dev).to(torch.uint8)
    unit = torch.pow(torch.tensor(2.0, dtype=F64), s.cpu().to(F64) - 127).repeat_interleave(32, 2)
    if kind == "mxfp8":
        q = torch.randn((E, rows, cols), generator=g, device=dev).to(torch.float8_e4m3fn)
        return q.view(torch.uint8), s, q.cpu().to(F64) * unit
    q = torch.randint(0, 256, (E, rows, cols // 2), generator=g, device=dev, dtype=torch.int32).to(torch.uint8)
    grid = torch.tensor(GRID, dtype=F64) / 3
    c = q.cpu().long()
    # the codes' values over three are what about one standard deviation is: halve the scales instead
    v = torch.stack((grid[c & 15], grid[c >> 4]), -1).flatten(2) * 3
    return q, s, v * unit


def layer64(x, z, bias, v1, v2, k, gate, renorm, scale, limit):
    ids, w = choose64(z, bias, k, gate, renorm, scale)
    x = x.cpu().to(F64)
    T, H = x.shape
    I = v2.shape[2]
    out, size = torch.zeros((T, H), dtype=F64), torch.zeros((T, H), dtype=F64)
    fine = 512 * 2.0 ** -24
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e < 0:
                continue
            c, big = v1[e] @ x[t], v1[e].abs() @ x[t].abs()
            g, u = c[:I], c[I:]
            if limit > 0:
                g, u = g.clamp(max=limit), u.clamp(-limit, limit)
            h = g * torch.sigmoid(g) * u
            dh = 2.0 ** -8 * h.abs() + fine * (1.1 * u.abs() * big[:I] + g.abs() * big[I:])
            out[t] += w[t, j] * (v2[e] @ h)
            size[t] += w[t, j] * (v2[e].abs() @ (dh + 2.0 ** -12 * h.abs()))
    return ids, w, out, size


def run(x, z, bias, w1, s1, w2, s2, k, gate, renorm, scale, kind, limit=0.0, ws=None, out=None):
    T, H = x.shape
    E = z.shape[1]
    I = w1.shape[1] // 2
    dev = x.device
    n = ptm.pt_moe_few_tokens_workspace_size(T, E, H, I, k)
    own = ws if ws is not None else torch.full((n + 256,), 0xFF, dtype=torch.uint8, device=dev)
    if ws is None:
        own[:4] = 0
    out = out if out is not None else torch.full((T, H), 7.0, dtype=torch.bfloat16, device=dev)
    ids = torch.full((T, k), 99, dtype=torch.int32, device=dev)
    w = torch.full((T, k), 7.0, device=dev)
    ptm.pt_moe_few_tokens(x, z, bias, w1, s1, w2, s2, out, ids, w, T, E, H, I, k,
                          ptm.PT_BF16 if z.dtype == torch.bfloat16 else ptm.PT_FP32, gate, renorm, scale, KINDS[kind],
                          workspace=own[:n], swiglu_limit=limit)
    torch.cuda.synchronize()
    if ws is None:
        assert own[n:].eq(0xFF).all()
    return out, ids, w


def check(x, z, bias, ops, k, gate, renorm, scale, kind, limit=0.0):
    (w1, s1, v1), (w2, s2, v2) = ops
    out, ids, w = run(x, z, bias, w1, s1, w2, s2, k, gate, renorm, scale, kind, limit)
    rids, rw, ref, size = layer64(x, z, bias, v1, v2, k, gate, renorm, scale, limit)
    assert torch.equal(ids.cpu(), rids)
    assert ((w.cpu().to(F64) - rw).abs() <= 80 * 2.0 ** -24 * rw.abs() + 1e-37).all()
    got = out.cpu().to(F64)
    assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + size + 1e-30).all()
    assert torch.linalg.norm(got - ref) <= 2.0 ** -7 * torch.linalg.norm(ref) + 1e-30
    return out


def make(dev, T, E, H, I, kind, seed, dtype=torch.float32):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((T, H), generator=g, device=dev).bfloat16()
    z = torch.randn((T, E), generator=g, device=dev).to(dtype)
    bias = 0.05 * torch.randn(E, generator=g, device=dev)
    return x, z, bias, (weights(g, E, 2 * I, H, kind), weights(g, E, H, I, kind))


# tokens, experts, hidden, inner, k: one token, more tokens than a tile's 16 for one expert, odd widths
SIZES = [(1, 1, 32, 32, 1), (1, 8, 96, 32, 3), (2, 60, 544, 160, 6), (5, 8, 288, 736, 2), (16, 4, 512, 256, 2),
         (17, 2, 160, 288, 2), (33, 3, 1056, 96, 2), (64, 2, 288, 160, 1), (64, 6, 352, 224, 4), (7, 256, 96, 64, 6),
         (3, 4, 2880, 64, 2), (3, 4, 64, 2880, 2), (64, 2, 4096, 64, 2), (9, 2, 64, 4128, 2)]


@pytest.mark.parametrize("T,E,H,I,k", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "mxfp8", "mxfp4"])
def test_layer(dev, T, E, H, I, k, kind):
    x, z, bias, ops = make(dev, T, E, H, I, kind, T * 13 + H + I)
    check(x, z, None, ops, k, 0, 1, 1.0, kind)
    check(x, z.bfloat16(), bias, ops, k, 1, int(k > 1), 2.5, kind)


@pytest.mark.parametrize("T,E,k", [(40, 256, 6), (64, 100, 16), (9, 600, 4)])
def test_many_experts(dev, T, E, k):
    """The choice of experts by several workgroups, and tokens without any."""
    x, z, bias, ops = make(dev, T, E, 96, 64, "mxfp8", T + E)
    check(x, z, bias, ops, k, 1, 1, 2.5, "mxfp8")
    z[T // 2:] = NINF
    check(x, z, None, ops, k, 0, 0, 1.0, "mxfp8")


@pytest.mark.parametrize("T,E,H,I,k", [(3, 4, 40, 24, 2), (20, 2, 72, 8, 2), (1, 3, 8, 16, 3), (18, 3, 264, 200, 2)])
def test_bf16_widths_in_eights(dev, T, E, H, I, k):
    x, z, _, ops = make(dev, T, E, H, I, "bf16", T + H)
    check(x, z, None, ops, k, 0, 0, 1.0, "bf16")


@pytest.mark.parametrize("kind", ["bf16", "mxfp8", "mxfp4"])
def test_widest(dev, kind):
    x, z, _, ops = make(dev, 5, 1, 16384, 32, kind, 3)
    check(x, z, None, ops, 1, 0, 1, 1.0, kind)
    x, z, _, ops = make(dev, 5, 1, 32, 16384, kind, 4)
    check(x, z, None, ops, 1, 0, 1, 1.0, kind)


@pytest.mark.parametrize("kind", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (40, 2, 2)])
def test_wide_rows_in_every_workgroup_size(dev, T, E, k, kind):
    """Few rows per expert and many: the workgroup's waves follow from both, a tile's share of them from the width."""
    for H, I in ((16384, 32), (32, 16384), (4096, 96)):
        x, z, _, ops = make(dev, T, E, H, I, kind, T + E + I)
        check(x, z, None, ops, k, 0, 1, 1.0, kind)


@pytest.mark.parametrize("kind", ["bf16", "mxfp8", "mxfp4"])
def test_clamped_swiglu(dev, kind):
    x, z, _, ops = make(dev, 6, 4, 128, 96, kind, 9)
    check(x * 4, z, None, ops, 2, 0, 1, 1.0, kind, limit=1.5)


@pytest.mark.parametrize("kind", ["bf16", "mxfp8", "mxfp4"])
def test_tokens_without_experts(dev, kind):
    x, z, _, ops = make(dev, 5, 6, 96, 64, kind, 11)
    z[1] = NINF
    z[3] = NINF
    z[3, 4] = 0.5
    out = check(x, z, None, ops, 3, 0, 1, 1.0, kind)
    assert out[1].eq(0).all()
    z[:] = NINF
    assert check(x, z, None, ops, 3, 0, 1, 1.0, kind).eq(0).all()


def test_a_nan_stays_with_its_token(dev):
    """A token or an expert that holds NaNs must not reach the tokens and experts that share its tiles."""
    for kind in ("bf16", "mxfp8", "mxfp4"):
        x, z, _, (a, b) = make(dev, 6, 4, 96, 64, kind, 17)
        z[:, 3] = NINF
        z[2, 3] = 5.0
        clean, _, _ = run(x, z, None, a[0], a[1], b[0], b[1], 2, 0, 1, 1.0, kind)
        bad = x.clone()
        bad[4, 5] = float("nan")
        out, _, _ = run(bad, z, None, a[0], a[1], b[0], b[1], 2, 0, 1, 1.0, kind)
        keep = [0, 1, 2, 3, 5]
        assert out[4].isnan().all() and torch.equal(out[keep], clean[keep])
        if kind == "mxfp4":
            s = b[1].clone()
            s[3, :, 1] = 255                             # E8M0 NaN
            out, _, _ = run(x, z, None, a[0], a[1], b[0], s, 2, 0, 1, 1.0, kind)
        else:
            w = b[0].clone()
            w[3, :, 40] = float("nan") if kind == "bf16" else 0x7F
            out, _, _ = run(x, z, None, a[0], a[1], w, b[1], 2, 0, 1, 1.0, kind)
        keep = [0, 1, 3, 4, 5]
        assert out[2].isnan().all() and torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("kind,byte", [("mxfp8", 0), ("mxfp8", 1), ("mxfp8", 60), ("mxfp4", 0), ("mxfp4", 60),
                                       ("mxfp8", 150), ("mxfp4", 150)])
def test_extreme_scale_bytes(dev, kind, byte):
    """Products that leave no room: w2 with one scale byte for all, FC1 as usual.  Below 2^-126 everything is zero."""
    x, z, _, (a, b) = make(dev, 3, 2, 64, 64, kind, 23)
    s = torch.full_like(b[1], byte)
    v = b[2] / torch.pow(torch.tensor(2.0, dtype=F64), b[1].cpu().to(F64) - 127).repeat_interleave(32, 2)
    v = v * 2.0 ** (byte - 127)
    out, _, _ = run(x, z, None, a[0], a[1], b[0], s, 2, 0, 1, 1.0, kind)
    _, _, ref, size = layer64(x, z, None, a[2], v, 2, 0, 1, 1.0, 0.0)
    # a weight under 2^-126 has steps of 2^-133 in bf16
    assert ((out.cpu().to(F64) - ref).abs() <= 2.0 ** -8 * ref.abs() + size + 64 * 2.0 ** -130).all()


def test_same_bits_again_and_on_dirty_memory(dev):
    for kind in KINDS:
        x, z, _, (a, b) = make(dev, 40, 5, 416, 352, kind, 29)
        args = (x, z, None, a[0], a[1], b[0], b[1], 3, 0, 1, 1.0, kind)
        first = run(*args)
        n = ptm.pt_moe_few_tokens_workspace_size(40, 5, 416, 352, 3)
        for fill in (0, 0xFF):
            ws = torch.full((n,), fill, dtype=torch.uint8, device=dev)
            for _ in range(3):
                again = run(*args, ws=ws)
                assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_a_token_alone_and_among_others(dev):
    """A token's result does not depend on who shares the call."""
    for kind in KINDS:
        x, z, _, (a, b) = make(dev, 40, 4, 288, 96, kind, 31)
        many, _, _ = run(x, z, None, a[0], a[1], b[0], b[1], 2, 0, 1, 1.0, kind)
        for t in (0, 17, 39):
            one, _, _ = run(x[t:t + 1].clone(), z[t:t + 1].clone(), None, a[0], a[1], b[0], b[1], 2, 0, 1, 1.0, kind)
            assert torch.equal(one[0], many[t])


def test_weights_past_four_gigabytes(dev):
    """The last expert of a tensor larger than 2^32 bytes."""
    E, H, I = 70, 4096, 2816                             # w1 is 70 * 5632 * 4096 * 2 = 3.2e9 bytes, w2 1.6e9
    E = 100                                              # 4.6e9
    w1 = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device=dev)
    w2 = torch.zeros((E, H, I), dtype=torch.bfloat16, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    w1[E - 1] = (torch.randn((2 * I, H), generator=g, device=dev) / 64).bfloat16()
    w2[E - 1] = (torch.randn((H, I), generator=g, device=dev) / 53).bfloat16()
    x = torch.randn((2, H), generator=g, device=dev).bfloat16()
    z = torch.zeros((2, E), device=dev)
    z[:, E - 1] = 9.0
    out, _, _ = run(x, z, None, w1, None, w2, None, 1, 0, 1, 1.0, "bf16")
    c = x.cpu().to(F64) @ w1[E - 1].cpu().to(F64).t()
    h = c[:, :I] * torch.sigmoid(c[:, :I]) * c[:, I:]
    ref = h @ w2[E - 1].cpu().to(F64).t()
    assert torch.linalg.norm(out.cpu().to(F64) - ref) <= 2.0 ** -7 * torch.linalg.norm(ref)


def test_streams_and_graph(dev):
    x, z, _, (a, b) = make(dev, 20, 8, 288, 160, "mxfp8", 37)
    ref, rids, rw = run(x, z, None, a[0], a[1], b[0], b[1], 3, 0, 1, 1.0, "mxfp8")
    n = ptm.pt_moe_few_tokens_workspace_size(20, 8, 288, 160, 3)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)
    out, ids, w = torch.zeros_like(ref), torch.zeros_like(rids), torch.zeros_like(rw)

    def go():
        ptm.pt_moe_few_tokens(x, z, None, a[0], a[1], b[0], b[1], out, ids, w, 20, 8, 288, 160, 3, ptm.PT_FP32, 0, 1, 1.0,
                              ptm.PT_MXFP8_E4M3, workspace=ws)

    def same():
        torch.cuda.synchronize()
        ok = torch.equal(out, ref) and torch.equal(ids, rids) and torch.equal(w, rw)
        out.zero_(), ids.zero_(), w.zero_()
        torch.cuda.synchronize()
        return ok

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        go()
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        graph.replay()
        assert same()
        go()
        assert same()


def test_two_streams_at_once(dev):
    """Calls on two streams, each with its own workspace and outputs."""
    x, z, _, (a, b) = make(dev, 30, 8, 512, 256, "bf16", 41)
    ref, _, _ = run(x, z, None, a[0], None, b[0], None, 2, 0, 1, 1.0, "bf16")
    n = ptm.pt_moe_few_tokens_workspace_size(30, 8, 512, 256, 2)
    sides = [torch.cuda.Stream() for _ in range(2)]
    own = [(torch.empty(n, dtype=torch.uint8, device=dev), torch.zeros_like(ref), torch.zeros((30, 2), dtype=torch.int32, device=dev),
            torch.zeros((30, 2), device=dev)) for _ in sides]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (ws, out, ids, w) in zip(sides, own):
            ptm.pt_moe_few_tokens(x, z, None, a[0], None, b[0], None, out, ids, w, 30, 8, 512, 256, 2, ptm.PT_FP32, 0, 1,
                                  1.0, ptm.PT_BF16, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o[1], ref) for o in own)
