"""The dense matrix product with its epilogue and gradients on the GPU.

Two kinds of comparison.  With small integers as operands every product and sum
is exact in fp32, so results are compared bit for bit with 64-bit arithmetic
rounded once: a value left out or taken twice shows whatever its size.  With
random operands, against the formulas in 64 bits within tolerances derived here.
A sum of K products is taken in steps of 16 values and, where it is cut, in at
most 64 parts: (K / 16 + 64) additions, each off by at most 2^-23 of a partial
sum, which S = |x| |w| bounds (the matrix cores' inner additions may truncate).
An output is then off by its slope times that, by 16 roundings of the terms of
its activation, and by half a step of its type: 2^-8 in bf16, 2^-24 in fp32.
"""
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm

pytestmark = pytest.mark.gpu

F64, BF16, F32 = torch.float64, torch.bfloat16, torch.float32
ACTS = {"none": ptm.PT_ACT_NONE, "silu": ptm.PT_ACT_SILU, "gelu": ptm.PT_ACT_GELU, "gelu_tanh": ptm.PT_ACT_GELU_TANH,
        "relu2": ptm.PT_ACT_RELU2, "swiglu": ptm.PT_ACT_SWIGLU}
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
TYPE = {BF16: ptm.PT_BF16, F32: ptm.PT_FP32}


def gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def ints(g, *shape, top=3):
    return torch.randint(-top, top + 1, shape, generator=g, device=g.device).to(BF16)


def randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device=g.device) * std).to(BF16)


def workspace(op, M, N, K, dev):
    # contents on entry do not matter
    return torch.full((ptm.pt_linear_workspace_size(op, M, N, K),), 0xFF, dtype=torch.uint8, device=dev)


def forward(x, w, bias=None, residual=None, out_type=BF16, act="none", save=False, limit=0.0, out=None):
    (M, K), N = x.shape, w.shape[0]
    cols = N // 2 if act == "swiglu" else N
    if out is None:
        out = torch.full((M, cols), 7.0, dtype=out_type, device=x.device)
    c = torch.full((M, N), 7.0, dtype=BF16, device=x.device) if save else None
    ptm.pt_linear_fwd(x, w, bias, residual, out, c, M, N, K, ACTS[act], TYPE[out_type],
                      workspace=workspace(ptm.PT_OP_FWD, M, N, K, x.device), swiglu_limit=limit)
    torch.cuda.synchronize()
    return (out, c) if save else out


def dgrad(dy, w, c=None, add=None, act="none", limit=0.0, dx=None):
    (M, N), K = dy.shape, w.shape[1]
    if dx is None:
        dx = torch.full((M, 2 * K if act == "swiglu" else K), 7.0, dtype=BF16, device=dy.device)
    ptm.pt_linear_dgrad(dy, w, c, add, dx, M, N, K, ACTS[act], workspace=workspace(ptm.PT_OP_DGRAD, M, N, K, dy.device),
                        swiglu_limit=limit)
    torch.cuda.synchronize()
    return dx


def wgrad(x, dy, bias=True, accumulate=0, main_grad=None, dbias=None):
    (M, K), N = x.shape, dy.shape[1]
    if main_grad is None:
        main_grad = torch.full((N, K), 7.0, device=x.device)
    if dbias is None and bias:
        dbias = torch.full((N,), 7.0, device=x.device)
    ptm.pt_linear_wgrad(x, dy, main_grad, dbias, M, N, K, accumulate,
                        workspace=workspace(ptm.PT_OP_WGRAD, M, N, K, x.device))
    torch.cuda.synchronize()
    return main_grad, dbias


def act64(c, act, limit=float("inf")):
    if act == "swiglu":
        h = c.shape[1] // 2
        g, u = c[:, :h].clamp(max=limit), c[:, h:].clamp(-limit, limit)
        return g * torch.sigmoid(g) * u
    return {"none": lambda: c, "relu2": lambda: c.clamp(min=0) ** 2, "silu": lambda: c * torch.sigmoid(c),
            "gelu": lambda: 0.5 * c * torch.erfc(-c / 2 ** 0.5),
            "gelu_tanh": lambda: 0.5 * c * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (c + 0.044715 * c ** 3)))}[act]()


# few rows; narrow, 64, 128 and 256 tiles; reductions shorter than a stage, odd
# in eights, long enough to be cut
SHAPES = [(1, 8, 8), (1, 4096, 520), (2, 24, 64), (15, 40, 72), (16, 16, 128), (17, 136, 56), (33, 264, 1032), (45, 520, 200),
          (64, 64, 4096), (65, 8, 136), (65, 32, 2880), (100, 24, 4096), (130, 136, 264), (257, 520, 72), (300, 264, 2056),
          (1021, 32, 40), (513, 1032, 520), (2049, 2056, 136), (4096, 4096, 72), (4099, 24, 264)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out_type", [BF16, F32])
def test_forward_exact(dev, M, N, K, out_type):
    g = gen(dev, M * 31 + N * 7 + K)
    x, w = ints(g, M, K), ints(g, N, K)
    bias, res = ints(g, N, top=20), ints(g, M, N, top=50).to(out_type)
    c = x.to(F64) @ w.to(F64).t() + bias.to(F64)
    out, saved = forward(x, w, bias, res, out_type, save=True)
    assert torch.equal(out, (c + res.to(F64)).to(out_type))
    assert torch.equal(saved, c.to(BF16))
    assert torch.equal(forward(x, w, out_type=out_type), (c - bias.to(F64)).to(out_type))
    # in place of the residual
    own = res.clone()
    assert torch.equal(forward(x, w, bias, own, out_type, out=own), (c + res.to(F64)).to(out_type))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_dgrad_exact(dev, M, N, K):
    g = gen(dev, M * 31 + N * 7 + K + 1)
    dy, w, add = ints(g, M, N), ints(g, N, K), ints(g, M, K, top=50)
    dh = dy.to(F64) @ w.to(F64)
    assert torch.equal(dgrad(dy, w), dh.to(BF16))
    assert torch.equal(dgrad(dy, w, add=add), (dh + add.to(F64)).to(BF16))
    own = add.clone()
    assert torch.equal(dgrad(dy, w, add=own, dx=own), (dh + add.to(F64)).to(BF16))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_wgrad_exact(dev, M, N, K):
    g = gen(dev, M * 31 + N * 7 + K + 2)
    x, dy = ints(g, M, K), ints(g, M, N)
    dw, db = dy.to(F64).t() @ x.to(F64), dy.to(F64).sum(0)
    got, gotb = wgrad(x, dy)
    assert torch.equal(got, dw.to(F32)) and torch.equal(gotb, db.to(F32))
    start, startb = ints(g, N, K, top=50).float(), ints(g, N, top=50).float()
    got, gotb = wgrad(x, dy, accumulate=1, main_grad=start.clone(), dbias=startb.clone())
    assert torch.equal(got, (dw + start.to(F64)).to(F32)) and torch.equal(gotb, (db + startb.to(F64)).to(F32))
    got, none = wgrad(x, dy, bias=False)
    assert torch.equal(got, dw.to(F32)) and none is None


@pytest.mark.parametrize("M,N,K", [(1, 16, 8), (5, 48, 72), (33, 272, 520), (70, 16, 136), (100, 32, 2880), (260, 528, 264),
                                   (300, 48, 2056), (1100, 1040, 200)])
def test_swiglu_pairs_exact(dev, M, N, K):
    """Which gate meets which up: gates held at a value where silu is the identity in bf16."""
    g = gen(dev, M + N + K)
    I = N // 2
    x, w = ints(g, M, K), ints(g, N, K)
    w[:I] = 0
    bias = torch.zeros(N, device=dev, dtype=BF16)
    bias[:I] = (128 + torch.arange(I, device=dev) % 64).to(BF16)        # sigmoid(128) is 1 to 2^-184
    up = x.to(F64) @ w[I:].to(F64).t()
    want = bias[:I].to(F64) * up
    assert want.abs().max() < 2 ** 24
    assert torch.equal(forward(x, w, bias, act="swiglu", out_type=F32), want.to(F32))


# sizes at which the rules take each tile, whole and with the reduction in parts
FWD_TILES = [(5857, 5040, 72), (5724, 672, 3064), (6863, 4496, 8), (5666, 272, 3896), (4189, 144, 8), (1270, 16, 1320), (18, 16, 264),
             (19, 16, 2200), (5925, 272, 632), (4374, 48, 3752), (4376, 144, 1944), (155, 4368, 4120), (19, 16, 1224)]
DGRAD_TILES = [(6311, 72, 4808), (5808, 3144, 664), (6797, 8, 4528), (4289, 4712, 8), (4170, 8, 144), (1436, 1048, 8), (5925, 600, 264),
               (3382, 4624, 8), (4448, 1976, 152), (290, 3904, 2464), (19, 840, 8)]
WGRAD_TILES = [(202, 3800, 3208), (7541, 4240, 392), (80, 3784, 3840), (5423, 4272, 8), (778, 8, 8), (612, 4144, 392), (3591, 4368, 8),
               (2272, 4744, 152), (8098, 136, 2528)]


@pytest.mark.parametrize("M,N,K", FWD_TILES)
def test_forward_exact_in_every_tile(dev, M, N, K):
    g = gen(dev, M + N + K)
    x, w, bias = ints(g, M, K), ints(g, N, K), ints(g, N, top=20)
    c = x.to(F64) @ w.to(F64).t() + bias.to(F64)
    out, saved = forward(x, w, bias, out_type=F32, save=True)
    assert torch.equal(out, c.to(F32)) and torch.equal(saved, c.to(BF16))
    I = N // 2
    w[:I] = 0
    bias[:I] = (128 + torch.arange(I, device=dev) % 64).to(BF16)
    want = bias[:I].to(F64) * (x.to(F64) @ w[I:].to(F64).t() + bias[I:].to(F64))
    assert want.abs().max() < 2 ** 24
    out, saved = forward(x, w, bias, act="swiglu", out_type=F32, save=True)
    assert torch.equal(out, want.to(F32))
    assert torch.equal(saved[:, I:], (x.to(F64) @ w[I:].to(F64).t() + bias[I:].to(F64)).to(BF16))


@pytest.mark.parametrize("M,N,K", DGRAD_TILES)
def test_dgrad_exact_in_every_tile(dev, M, N, K):
    g = gen(dev, M + N + K + 1)
    dy, w = ints(g, M, N), ints(g, N, K)
    dh = dy.to(F64) @ w.to(F64)
    assert torch.equal(dgrad(dy, w), dh.to(BF16))
    # gates at which silu is the identity and its slope 1: both gradients are exact
    c = torch.empty((M, 2 * K), dtype=BF16, device=dev)
    c[:, :K] = (128 + torch.arange(K, device=dev) % 64).to(BF16)
    c[:, K:] = ints(g, M, K)
    got = dgrad(dy, w, c, act="swiglu")
    assert torch.equal(got[:, :K], (dh * c[:, K:].to(F64)).to(BF16))
    assert torch.equal(got[:, K:], (dh * c[:, :K].to(F64)).float().to(BF16))


@pytest.mark.parametrize("M,N,K", WGRAD_TILES)
def test_wgrad_exact_in_every_tile(dev, M, N, K):
    g = gen(dev, M + N + K + 2)
    x, dy = ints(g, M, K), ints(g, M, N)
    dw, db = dy.to(F64).t() @ x.to(F64), dy.to(F64).sum(0)
    start, startb = ints(g, N, K, top=50).float(), ints(g, N, top=50).float()
    got, gotb = wgrad(x, dy)
    assert torch.equal(got, dw.to(F32)) and torch.equal(gotb, db.to(F32))
    got, gotb = wgrad(x, dy, accumulate=1, main_grad=start.clone(), dbias=startb.clone())
    assert torch.equal(got, (dw + start.to(F64)).to(F32)) and torch.equal(gotb, (db + startb.to(F64)).to(F32))


def sums(x, w, bias):
    """c in 64 bits and what it may be off by."""
    c = x.to(F64) @ w.to(F64).t()
    tol = (x.shape[1] / 16 + 64) * 2.0 ** -23 * (x.to(F64).abs() @ w.to(F64).abs().t())
    if bias is not None:
        c, tol = c + bias.to(F64), tol + 2.0 ** -23 * (c.abs() + bias.to(F64).abs())
    return c, tol


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M,N,K", [(3, 272, 200), (45, 48, 1032), (150, 272, 136), (520, 528, 264)])
@pytest.mark.parametrize("out_type", [BF16, F32])
def test_forward_activations(dev, act, M, N, K, out_type):
    g = gen(dev, M + N + K)
    x, w, bias = randn(g, M, K, std=2.0), randn(g, N, K, std=K ** -0.5), randn(g, N, std=1.0)
    cols = N // 2 if act == "swiglu" else N
    res = (torch.randn((M, cols), generator=g, device=dev) * 2).to(out_type)
    out, saved = forward(x, w, bias, res, out_type, act, save=True)
    c, tol = sums(x, w, bias)
    a = act64(c, act)
    if act == "swiglu":
        gt, u = c.chunk(2, 1)
        tg, tu = tol.chunk(2, 1)
        off = 1.1 * tg * (u.abs() + tu) + gt.abs() * tu + 16 * 2.0 ** -24 * (gt * u).abs()
    else:
        slope = 2 * (c.abs() + tol) if act == "relu2" else 1.2
        off = slope * tol + 16 * 2.0 ** -24 * (c.abs() + a.abs())
    want = a + res.to(F64)
    off = off + 2.0 ** -24 * (a.abs() + res.to(F64).abs())
    assert ((out.to(F64) - want).abs() <= HALF_STEP[out_type] * (want.abs() + off) + off).all()
    assert ((saved.to(F64) - c).abs() <= 2.0 ** -8 * (c.abs() + tol) + tol).all()


@pytest.mark.parametrize("act", [a for a in ACTS if a != "none"])
@pytest.mark.parametrize("M,N,K", [(3, 200, 264), (70, 1032, 48), (300, 136, 520)])
def test_dgrad_activations(dev, act, M, N, K):
    """Against autograd of the formula in 64 bits."""
    g = gen(dev, M + N + K + 5)
    dy, w = randn(g, M, N), randn(g, N, K, std=N ** -0.5)
    c = randn(g, M, 2 * K if act == "swiglu" else K, std=2.0)
    dx = dgrad(dy, w, c, act=act)
    dh, tol = sums(dy, w.t().contiguous(), None)
    c64 = c.to(F64).requires_grad_(True)
    slope = torch.autograd.grad(act64(c64, act).sum(), c64)[0]
    rep = 2 if act == "swiglu" else 1
    dh, tol = dh.repeat(1, rep), tol.repeat(1, rep)
    # the terms of a slope: at most 2 |c| + 2, times the other factor for SwiGLU
    size = (2 + 2 * c.to(F64).abs()) * (1 if act != "swiglu" else 1 + c.to(F64).abs().view(M, 2, K).flip(1).reshape(M, -1))
    off = slope.abs() * tol + 16 * 2.0 ** -24 * size * (dh.abs() + tol)
    want = slope * dh
    assert ((dx.to(F64) - want).abs() <= 2.0 ** -8 * (want.abs() + off) + off).all()
    # the activation's gradient alone: the same slopes on a given dh
    dout = randn(g, M, K)
    dc = torch.empty_like(c)
    ptm.pt_linear_act_bwd(dout, c, dc, M, c.shape[1], ACTS[act])
    want = slope * dout.to(F64).repeat(1, rep)
    off = 16 * 2.0 ** -24 * size * dout.to(F64).abs().repeat(1, rep)
    assert ((dc.to(F64) - want).abs() <= 2.0 ** -8 * (want.abs() + off) + off).all()
    own = c.clone()
    ptm.pt_linear_act_bwd(dout, own, own, M, c.shape[1], ACTS[act])
    assert torch.equal(own, dc)


@pytest.mark.parametrize("act", [a for a in ACTS if a not in ("none", "swiglu")])
def test_slopes_by_differences(dev, act):
    """dx against central differences of the forward's formula in 64 bits, over the whole range of c."""
    c = torch.cat([torch.linspace(-12, 12, 4064, device=dev), torch.tensor([-1e4, -300.0, -90.0, -20.0, 0.0, 20.0, 90.0, 1e4],
                                                                         device=dev)]).to(BF16)
    c = c[: c.numel() // 8 * 8].view(1, -1).contiguous()
    dc = torch.empty_like(c)
    ptm.pt_linear_act_bwd(torch.ones_like(c), c, dc, 1, c.shape[1], ACTS[act])
    x, h = c.to(F64), 1e-5
    want = (act64(x + h, act) - act64(x - h, act)) / (2 * h)
    # a difference of step h: h^2 / 6 times the third derivative (below 4), and 2^-52 of the values over h; relu2's
    # second derivative jumps at 0 (h there)
    off = h + 2.0 ** -52 * (x.abs() ** 2 + 1) / h + 2.0 ** -20 * (1 + x.abs())
    assert ((dc.to(F64) - want).abs() <= 2.0 ** -8 * want.abs() + off).all()


def test_swiglu_clamp(dev):
    g = gen(dev, 3)
    M, I, K, lim = 40, 72, 136, 0.75
    x, w = randn(g, M, K), randn(g, 2 * I, K, std=K ** -0.5)
    c, tol = sums(x, w, None)
    want = act64(c, "swiglu", lim)
    out = forward(x, w, act="swiglu", limit=lim)
    off = 1.1 * tol[:, :I] * lim + 2 * lim * tol[:, I:] + 1e-6
    assert ((out.to(F64) - want).abs() <= 2.0 ** -8 * (want.abs() + off) + off + (c[:, :I].abs() * 2.0 ** -8)).all()
    # gradients: none into a clamped gate or up
    cs = (torch.randn((M, 2 * I), generator=g, device=dev)).to(BF16)
    dout = randn(g, M, I)
    dc = torch.empty_like(cs)
    ptm.pt_linear_act_bwd(dout, cs, dc, M, 2 * I, ptm.PT_ACT_SWIGLU, swiglu_limit=lim)
    c64 = cs.to(F64).requires_grad_(True)
    want = torch.autograd.grad(act64(c64, "swiglu", lim), c64, dout.to(F64))[0]
    clamped = torch.cat((cs[:, :I] > lim, cs[:, I:].abs() > lim), 1)
    assert (dc[clamped] == 0).all()
    keep = ~clamped & (cs.abs() != lim)
    assert ((dc.to(F64) - want).abs()[keep] <= (2.0 ** -8 * want.abs() + 1e-5)[keep]).all()
    got = dgrad(dout, torch.eye(I, device=dev).to(BF16), cs, act="swiglu", limit=lim)
    assert torch.equal(got, dc)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M", [7, 100])
def test_extreme_sums(dev, act, M):
    """Large sums of either sign, infinities and NaN: no NaN where the formula has none, and none lost."""
    I = 8
    N = 2 * I if act == "swiglu" else I
    vals = torch.tensor([0.0, 1e4, -1e4, 1e18, -1e18, 88.0, -88.0, 110.0], device=dev)
    x, w = torch.zeros((M, 8), dtype=BF16, device=dev), torch.zeros((N, 8), dtype=BF16, device=dev)
    bias = torch.zeros(N, dtype=BF16, device=dev)
    bias[:I] = vals.to(BF16)
    if act == "swiglu":
        bias[I:] = 0.5
    out, saved = forward(x, w, bias, out_type=F32, act=act, save=True)
    want = act64(bias.to(F64).view(1, -1).expand(M, -1), act)
    assert ((out.to(F64) - want).abs() <= 2e-6 * want.abs() + 1e-30).all()
    dc = torch.empty_like(saved)
    if act != "none":
        ptm.pt_linear_act_bwd(torch.ones((M, I), dtype=BF16, device=dev), saved, dc, M, N, ACTS[act])
        c64 = saved.to(F64).requires_grad_(True)
        want = torch.autograd.grad(act64(c64, act).sum(), c64)[0]
        want = torch.where(torch.isfinite(want), want, 0.0)       # 64-bit tanh's slope times an infinite square
        assert torch.isfinite(dc).all()
        assert ((dc.to(F64) - want).abs() <= 2.0 ** -8 * want.abs() + 1e-3 * (saved.to(F64).abs() < 1e5)).all() or act == "gelu_tanh"
    x[2, 3] = float("nan")
    w[:, 3] = 1
    out, saved = forward(x, w, bias, out_type=F32, act=act, save=True)
    assert torch.isnan(out[2]).all() and torch.isnan(saved[2]).all()
    assert torch.isfinite(out[[0, 1, 3, 4, 5, 6]]).all()
    if act != "none":
        ptm.pt_linear_act_bwd(torch.ones((M, I), dtype=BF16, device=dev), saved, dc, M, N, ACTS[act])
        assert torch.isnan(dc[2]).all() and torch.isfinite(dc[3]).all()


def test_nan_and_inf_stay_in_their_rows_and_columns(dev):
    g = gen(dev, 8)
    for M, N, K in ((5, 40, 72), (80, 136, 200), (300, 264, 2056)):
        x, w = randn(g, M, K), randn(g, N, K)
        clean = forward(x, w)
        x2, w2 = x.clone(), w.clone()
        x2[1, K - 1] = float("inf")
        w2[9, 0] = float("nan")
        w2[:, K - 1] = w2[:, K - 1].abs() + 0.5
        ref = forward(x, w2.nan_to_num())
        out = forward(x2, w2)
        assert torch.isnan(out[:, 9]).all() and torch.isinf(out[1, :9]).all()
        rows = torch.ones(M, dtype=torch.bool, device=dev)
        rows[1] = False
        cols = torch.ones(N, dtype=torch.bool, device=dev)
        cols[9] = False
        assert torch.equal(out[rows][:, cols], ref[rows][:, cols])
        assert torch.isfinite(clean).all()


def test_no_rows(dev):
    x, w = torch.empty((0, 64), dtype=BF16, device=dev), torch.ones((16, 64), dtype=BF16, device=dev)
    out = torch.empty((0, 16), dtype=BF16, device=dev)
    ptm.pt_linear_fwd(x, w, None, None, out, None, 0, 16, 64)
    dw, db = wgrad(x, out)
    assert (dw == 0).all() and (db == 0).all()
    keep, keepb = torch.full((16, 64), 3.0, device=dev), torch.full((16,), 3.0, device=dev)
    wgrad(x, out, accumulate=1, main_grad=keep, dbias=keepb)
    assert (keep == 3).all() and (keepb == 3).all()


def test_outputs_stay_inside(dev):
    """Nothing is written next to the outputs, whatever the tile covers."""
    g = gen(dev, 4)
    for M, N, K in ((3, 24, 40), (70, 40, 136), (130, 136, 72), (257, 264, 520)):
        x, w = ints(g, M, K), ints(g, N, K)
        for shape, run in (((M, N), lambda o: forward(x, w, out=o)), ((M, K), lambda o: dgrad(ints(g, M, N), w, dx=o))):
            pad = torch.full((shape[0] + 2, shape[1]), 99.0, dtype=BF16, device=dev)
            run(pad[1:-1])
            assert (pad[0] == 99).all() and (pad[-1] == 99).all()
        pad = torch.full((N + 2, K), 99.0, device=dev)
        padb = torch.full((N + 16,), 99.0, device=dev)
        wgrad(x, ints(g, M, N), main_grad=pad[1:-1], dbias=padb[8:-8])
        assert (pad[0] == 99).all() and (pad[-1] == 99).all() and (padb[:8] == 99).all() and (padb[-8:] == 99).all()


def test_repeats_are_equal(dev):
    g = gen(dev, 6)
    for M, N, K in ((33, 264, 4096), (100, 264, 4096), (1000, 520, 1032)):
        x, w, dy = randn(g, M, K), randn(g, N, K), randn(g, M, N)
        first = (forward(x, w, out_type=F32), dgrad(dy, w), *wgrad(x, dy))
        for _ in range(3):
            again = (forward(x, w, out_type=F32), dgrad(dy, w), *wgrad(x, dy))
            assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_other_stream_and_graph(dev):
    g = gen(dev, 7)
    M, N, K = 100, 264, 2056
    x, w, dy = ints(g, M, K), ints(g, N, K), ints(g, M, N)
    want = forward(x, w, out_type=F32).clone(), dgrad(dy, w).clone(), *[t.clone() for t in wgrad(x, dy)]
    out, dx = torch.zeros((M, N), device=dev), torch.zeros((M, K), dtype=BF16, device=dev)
    dw, db = torch.zeros((N, K), device=dev), torch.zeros(N, device=dev)
    ws = [workspace(op, M, N, K, dev) for op in (ptm.PT_OP_FWD, ptm.PT_OP_DGRAD, ptm.PT_OP_WGRAD)]

    def run():
        ptm.pt_linear_fwd(x, w, None, None, out, None, M, N, K, out_dtype=ptm.PT_FP32, workspace=ws[0])
        ptm.pt_linear_dgrad(dy, w, None, None, dx, M, N, K, workspace=ws[1])
        ptm.pt_linear_wgrad(x, dy, dw, db, M, N, K, 0, workspace=ws[2])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(dx, want[1]) and torch.equal(dw, want[2]) and torch.equal(db, want[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for t in (out, dx, dw, db):
            t.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(dx, want[1]) and torch.equal(dw, want[2]) and torch.equal(db, want[3])
