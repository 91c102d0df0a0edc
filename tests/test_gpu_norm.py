"""Residual RMS norm on the GPU against the formulas in 64 bits.

Tolerances, derived: the stream is one rounding of an exact sum, so it is
compared bit for bit.  rstd: a sum of `cols` squares in a tree at most 40 deep
(relative error 40 * 2^-24, halved by the square root) and three roundings:
24 * 2^-24 < 2e-6.  y is v = h rstd w (three fp32 roundings more) rounded to
bf16: 2^-8 + 3e-6.  A code is v over its scale rounded to E4M3: 2^-4, or
half of the smallest step 2^-9 below 2^-6.
"""
import numpy as np
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm

pytestmark = pytest.mark.gpu

F64 = torch.float64
CODES = {"none": ptm.PT_BF16, "mxfp8": ptm.PT_MXFP8_E4M3, "rows": ptm.PT_FP8_E4M3_ROWWISE}
STREAM = {"bf16": (ptm.PT_BF16, torch.bfloat16), "f32": (ptm.PT_FP32, torch.float32)}


def gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def inputs(dev, rows, cols, stream, seed):
    g = gen(dev, seed)
    x = torch.randn((rows, cols), generator=g, device=dev).bfloat16()
    res = (torch.randn((rows, cols), generator=g, device=dev) * 3).to(STREAM[stream][1])
    w = (1 + 0.2 * torch.randn(cols, generator=g, device=dev)).bfloat16()
    return x, res, w


def forward(x, res, w, stream, codes, eps=1e-5, with_y=True, residual_out=None):
    rows, cols = x.shape
    dev, st = x.device, STREAM[stream]
    out = {"h": residual_out if residual_out is not None else torch.full((rows, cols), 7.0, dtype=st[1], device=dev),
           "y": torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=dev) if with_y else None,
           "rstd": torch.full((rows,), 7.0, device=dev), "q": None, "scales": None}
    if codes != "none":
        out["q"] = torch.full((rows, cols), 0xEE, dtype=torch.uint8, device=dev)
        out["scales"] = (torch.full((rows, cols // 32), 0xEE, dtype=torch.uint8, device=dev) if codes == "mxfp8"
                         else torch.full((rows,), 7.0, device=dev))
    ptm.pt_rmsnorm_fwd(x, res, w, out["h"], out["y"], out["q"], out["scales"], out["rstd"], rows, cols, eps, st[0],
                       CODES[codes])
    torch.cuda.synchronize()
    return out


def check_forward(x, res, w, stream, codes, got, eps=1e-5):
    t = STREAM[stream][1]
    h = (x.float() + res.float()).to(t) if res is not None else x.to(t)
    assert torch.equal(got["h"], h)
    h = h.to(F64)
    rstd = (h.square().mean(1) + eps).pow(-0.5)
    assert ((got["rstd"].to(F64) - rstd).abs() <= 2e-6 * rstd).all()
    v = h * rstd[:, None] * w.to(F64)
    if got["y"] is not None:
        assert ((got["y"].to(F64) - v).abs() <= (2.0 ** -8 + 3e-6) * v.abs() + 2.0 ** -134).all()
    if codes == "none":
        return
    deq = got["q"].view(torch.float8_e4m3fn).to(F64)
    if codes == "mxfp8":
        amax = v.unflatten(1, (-1, 32)).abs().amax(2)
        e = torch.floor(torch.log2(amax)).clamp(min=-127 + 8) - 8
        e = torch.where(amax > 0, e, torch.full_like(e, -127))
        have = got["scales"].to(F64) - 127
        # next to a power of two the amax may round across it
        edge = ((torch.log2(amax) - torch.round(torch.log2(amax))).abs() < 6e-6) & ((have - e).abs() == 1)
        assert (((have == e) | edge)).all()
        unit = torch.pow(torch.full_like(have, 2.0), have).repeat_interleave(32, 1)
    else:
        amax = v.abs().amax(1)
        factor = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        assert ((got["scales"].to(F64) - factor).abs() <= 4e-6 * factor).all()
        unit = got["scales"].to(F64)[:, None]
    want = (v / unit).clamp(-448, 448)
    assert ((deq - want).abs() <= (2.0 ** -4 + 1e-5) * want.abs() + 2.0 ** -10).all()


SHAPES = [(1, 8), (1, 4096), (3, 40), (5, 2880), (64, 2880), (7, 5056), (33, 288), (2, 2048), (2, 2056), (9, 6144),
          (2, 8192), (2, 8224), (3, 16384), (1, 32768), (1030, 544)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("codes", ["none", "mxfp8", "rows"])
def test_forward(dev, rows, cols, stream, codes):
    if codes == "mxfp8" and cols % 32:
        pytest.skip("blocks of 32")
    x, res, w = inputs(dev, rows, cols, stream, rows * 7 + cols)
    check_forward(x, res, w, stream, codes, forward(x, res, w, stream, codes))


@pytest.mark.parametrize("codes", ["none", "mxfp8", "rows"])
def test_optional_operands_and_in_place(dev, codes):
    x, res, w = inputs(dev, 6, 320, "f32", 5)
    whole = forward(x, res, w, "f32", codes)
    # the stream updated in place
    own = res.clone()
    got = forward(x, own, w, "f32", codes, residual_out=own)
    check_forward(x, res, w, "f32", codes, got)
    # no residual: the norm of x alone, in either stream type
    for stream in ("bf16", "f32"):
        check_forward(x, None, w, stream, codes, forward(x, None, w, stream, codes))
    if codes != "none":
        bare = forward(x, res, w, "f32", codes, with_y=False)
        assert torch.equal(bare["q"], whole["q"]) and torch.equal(bare["scales"], whole["scales"])
    q, s = whole["q"], whole["scales"]
    y = torch.empty_like(whole["y"])
    ptm.pt_rmsnorm_fwd(x, res, w, whole["h"], y, q, s, None, 6, 320, 1e-5, ptm.PT_FP32, CODES[codes])
    assert torch.equal(y, whole["y"])


@pytest.mark.parametrize("codes", ["none", "mxfp8", "rows"])
def test_zero_rows_tiny_huge_and_nan(dev, codes):
    x, res, w = inputs(dev, 6, 256, "f32", 9)
    x[0], res[0] = 0, 0
    x[1], res[1] = x[1] * 1e-30, res[1] * 1e-20           # all below sqrt(eps): v is h / sqrt(eps)
    x[2], res[2] = 0, res[2] * 1e15
    x[4, 17] = float("nan")
    x[5, 200] = float("inf")
    got = forward(x, res, w, "f32", codes)
    ok = slice(0, 4)
    check_forward(x[ok], res[ok], w, "f32", codes, {k: v[ok] if v is not None else None for k, v in got.items()})
    assert got["y"][0].eq(0).all() and got["y"][4].isnan().all() and got["y"][5].isnan().any()
    if codes != "none":
        deq = got["q"].view(torch.float8_e4m3fn).float()
        assert deq[0].eq(0).all() and deq[4].isnan().all()
        assert torch.equal(deq[5].isnan(), got["y"][5].isnan()) or deq[5].isnan().all()


def test_rows_do_not_touch_their_neighbours(dev):
    # every output has guard rows before and after
    x, res, w = inputs(dev, 5, 416, "bf16", 3)
    big = {n: torch.full((9, 416), 3.0, dtype=torch.bfloat16, device=dev) for n in ("h", "y")}
    q = torch.full((9, 416), 0xEE, dtype=torch.uint8, device=dev)
    s = torch.full((9, 13), 0xEE, dtype=torch.uint8, device=dev)
    ptm.pt_rmsnorm_fwd(x, res, w, big["h"][2:7], big["y"][2:7], q[2:7], s.view(-1)[26:91], None, 5, 416, 1e-5,
                       ptm.PT_BF16, ptm.PT_MXFP8_E4M3)
    for t, v in ((big["h"], 3.0), (big["y"], 3.0), (q, 0xEE), (s, 0xEE)):
        assert t[:2].eq(v).all() and t[7:].eq(v).all()


def backward(dy, s, w, rstd, dres, stream, accumulate=0, dweight=None, in_place=False):
    rows, cols = dy.shape
    ds = dres if in_place else torch.full((rows, cols), 7.0, dtype=STREAM[stream][1], device=dy.device)
    dw = dweight if dweight is not None else torch.full((cols,), 7.0, device=dy.device)
    n = ptm.pt_rmsnorm_workspace_size(rows, cols)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=dy.device)
    ptm.pt_rmsnorm_bwd(dy, s, w, rstd, dres, ds, dw, rows, cols, STREAM[stream][0], accumulate, workspace=ws[:n] if n else None)
    torch.cuda.synchronize()
    assert ws[n:].eq(0xFF).all()
    return ds, dw


def backward_reference(dy, s, w, rstd, dres):
    """ds and dweight in 64 bits, and the sizes of what is summed in each."""
    dy, s, w, r = (t.to(F64) for t in (dy, s, w, rstd[:, None]))
    xhat, g = s * r, dy * w
    mean = (g * xhat).mean(1, keepdim=True)
    ds = r * (g - xhat * mean)
    big = r * (g.abs() + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True))
    if dres is not None:
        ds, big = ds + dres.to(F64), big + dres.to(F64).abs()
    return ds, big, (dy * xhat).sum(0), (dy * xhat).abs().sum(0)


BWD_SHAPES = [(1, 8), (1, 4096), (2, 40), (8, 2880), (9, 2880), (65, 288), (517, 416), (1024, 64), (1500, 96),
              (40, 5056), (10, 8224), (12, 32768)]


@pytest.mark.parametrize("rows,cols", BWD_SHAPES)
@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("with_dres", [True, False])
def test_backward(dev, rows, cols, stream, with_dres):
    x, s, w = inputs(dev, rows, cols, stream, rows + cols)
    g = gen(dev, 77)
    dy = (torch.randn((rows, cols), generator=g, device=dev) * 1e-2).bfloat16()
    dres = (torch.randn((rows, cols), generator=g, device=dev) * 1e-2).to(s.dtype) if with_dres else None
    rstd = torch.rsqrt(s.float().square().mean(1) + 1e-5)
    ds, dw = backward(dy, s, w, rstd, dres, stream)
    ref, big, rdw, bdw = backward_reference(dy, s, w, rstd, dres)
    # fp32 arithmetic on each term (the mean's tree is at most 40 deep, as in the forward) and the output's rounding
    half = torch.finfo(s.dtype).eps / 2
    assert ((ds.to(F64) - ref).abs() <= half * ref.abs() + 64 * 2.0 ** -24 * big).all()
    # a column's sum: at most `rows` additions one after another, and two roundings a term
    assert ((dw.to(F64) - rdw).abs() <= (rows + 4) * 2.0 ** -24 * bdw + 1e-30).all()
    # again, in place of dres and added to what is there: the same bits, one more addition
    ds2, dw2 = backward(dy, s, w, rstd, dres.clone() if with_dres else None, stream, 1, torch.full_like(dw, 0.5),
                        in_place=with_dres)
    assert torch.equal(ds2, ds) and ((dw2 - (dw + 0.5)).abs() <= 2.0 ** -22).all()


def test_backward_without_weight_gradient_and_without_rows(dev):
    x, s, w = inputs(dev, 20, 96, "f32", 1)
    dy = x * 0.01
    rstd = torch.rsqrt(s.square().mean(1) + 1e-5)
    ds, _ = backward(dy, s, w, rstd, None, "f32")
    bare = torch.empty_like(ds)
    ptm.pt_rmsnorm_bwd(dy, s, w, rstd, None, bare, None, 20, 96, ptm.PT_FP32, 0)
    assert torch.equal(bare, ds)
    dw = torch.full((96,), 2.0, device=dev)
    e = s[:0]
    ptm.pt_rmsnorm_bwd(e.bfloat16(), e, w, rstd[:0], None, e, dw, 0, 96, ptm.PT_FP32, 1)
    assert dw.eq(2).all()
    ptm.pt_rmsnorm_bwd(e.bfloat16(), e, w, rstd[:0], None, e, dw, 0, 96, ptm.PT_FP32, 0)
    assert dw.eq(0).all()


def test_gradient_against_differences(dev):
    """The kernels' gradients along a direction against central differences of the definition in 64 bits."""
    rows, cols, eps = 12, 352, 1e-5
    x, s, w = inputs(dev, rows, cols, "f32", 21)
    g = gen(dev, 22)
    dy = torch.randn((rows, cols), generator=g, device=dev).bfloat16()
    dres = torch.randn((rows, cols), generator=g, device=dev)
    rstd = forward(torch.zeros_like(x), s, w, "f32", "none", eps)["rstd"]
    ds, dw = backward(dy, s, w, rstd, dres, "f32")
    du, dv = (torch.randn(t.shape, generator=g, device=dev, dtype=F64) for t in (s, w))

    def loss(t):
        h, ww = s.to(F64) + t * du, w.to(F64) + t * dv
        y = h * (h.square().mean(1, keepdim=True) + eps).pow(-0.5) * ww
        return ((y * dy.to(F64)).sum() + (h * dres.to(F64)).sum()).item()

    t = 1e-5
    numeric = (loss(t) - loss(-t)) / (2 * t)
    ours = ((ds.to(F64) * du).sum() + (dw.to(F64) * dv).sum()).item()
    # differences: t^2 times a third derivative of order one per element, and 2^-52 of the loss over t;
    # the kernels' terms: 64 roundings of 2^-24 each on what backward_reference calls big
    _, big, _, bdw = backward_reference(dy, s, w, rstd, dres)
    slack = 64 * 2.0 ** -24 * ((big * du.abs()).sum() + (bdw * dv.abs()).sum()).item() + 1e-4
    assert abs(numeric - ours) <= slack


def test_elements_past_32_bits(dev):
    """More than 2^31 elements: the last rows like a call of their own, and a weight gradient that only they feed."""
    rows, cols, k = 65600, 32768, 40
    x, s, w = inputs(dev, k, cols, "bf16", 41)
    big = {n: torch.zeros((rows, cols), dtype=torch.bfloat16, device=dev) for n in ("x", "s", "h", "y")}
    big["x"][-k:], big["s"][-k:] = x, s
    q = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    scales, rstd = torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev), torch.empty(rows, device=dev)
    ptm.pt_rmsnorm_fwd(big["x"], big["s"], w, big["h"], big["y"], q, scales, rstd, rows, cols, 1e-5, ptm.PT_BF16,
                       ptm.PT_MXFP8_E4M3)
    ref = forward(x, s, w, "bf16", "mxfp8")
    for got, want in ((big["h"], "h"), (big["y"], "y"), (q, "q"), (scales, "scales"), (rstd, "rstd")):
        assert torch.equal(got[-k:], ref[want])
    assert big["y"][:-k].eq(0).all() and q[:-k].eq(0).all()
    dy = big["x"]                                        # zero but for the last rows
    n = ptm.pt_rmsnorm_workspace_size(rows, cols)
    ds, dw = big["y"], torch.empty(cols, device=dev)
    ptm.pt_rmsnorm_bwd(dy, big["h"], w, rstd, None, ds, dw, rows, cols, ptm.PT_BF16, 0,
                       workspace=torch.empty(n, dtype=torch.uint8, device=dev))
    rds, rdw = backward(x, ref["h"], w, ref["rstd"], None, "bf16")
    assert torch.equal(ds[-k:], rds) and ds[:-k].eq(0).all()
    # the same terms in another order: at most k additions, each off by 2^-24 of the sum of their sizes
    _, _, _, size = backward_reference(x, ref["h"], w, ref["rstd"], None)
    assert ((dw.to(F64) - rdw.to(F64)).abs() <= 2 * (k + 4) * 2.0 ** -24 * size).all()


def test_streams_and_graph(dev):
    """On a side stream, and captured: every replay gives the eager bits."""
    x, s, w = inputs(dev, 100, 2880, "bf16", 31)
    dy = x * 0.01
    eager = forward(x, s, w, "bf16", "mxfp8")
    ds, dw = backward(dy, eager["h"], w, eager["rstd"], s, "bf16")
    side = torch.cuda.Stream()
    out = {k: torch.zeros_like(v) for k, v in eager.items()}
    ds2, dw2 = torch.zeros_like(ds), torch.zeros_like(dw)
    ws = torch.empty(ptm.pt_rmsnorm_workspace_size(100, 2880), dtype=torch.uint8, device=dev)

    def run():
        ptm.pt_rmsnorm_fwd(x, s, w, out["h"], out["y"], out["q"], out["scales"], out["rstd"], 100, 2880, 1e-5,
                           ptm.PT_BF16, ptm.PT_MXFP8_E4M3)
        ptm.pt_rmsnorm_bwd(dy, out["h"], w, out["rstd"], s, ds2, dw2, 100, 2880, ptm.PT_BF16, 0, workspace=ws)

    def same():
        torch.cuda.synchronize()
        ok = all(torch.equal(out[k], eager[k]) for k in eager) and torch.equal(ds2, ds) and torch.equal(dw2, dw)
        for t in (*out.values(), ds2, dw2):
            t.zero_()
        torch.cuda.synchronize()
        return ok

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        run()
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        graph.replay()
        assert same()
        run()                                            # the program's own eager work between replays
        assert same()
