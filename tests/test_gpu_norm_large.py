"""RMS norm where a team takes several rows one after another, and where a call
is large enough for its rows to go past the caches: random data in every row,
against 64 bits (on the GPU), and against calls of a part of the rows.

Tolerances as in test_gpu_norm, but for the weight gradient, whose additions
are counted: a term has two roundings and passes through at most ceil(rows /
parts) additions of a part's rows, 3 of a workgroup's teams, ceil(parts / 128)
and 7 of the join of the parts, and one of what is accumulated to.
"""
import math

import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm
from test_gpu_norm import F64, STREAM, backward, backward_reference, check_forward, forward, gen, inputs

pytestmark = pytest.mark.gpu


def check_backward(dy, s, w, rstd, dres, stream):
    rows, cols = dy.shape
    ds, dw = backward(dy, s, w, rstd, dres, stream)
    ref, big, rdw, bdw = backward_reference(dy, s, w, rstd, dres)
    half = torch.finfo(s.dtype).eps / 2
    assert ((ds.to(F64) - ref).abs() <= half * ref.abs() + 64 * 2.0 ** -24 * big).all()
    del ref, big
    parts = max(ptm.pt_rmsnorm_workspace_size(rows, cols) // (4 * cols), 1)
    steps = math.ceil(rows / parts) + math.ceil(parts / 128) + 13
    assert ((dw.to(F64) - rdw).abs() <= steps * 2.0 ** -24 * bdw + 1e-30).all()
    return ds, dw


def gradients(dev, rows, cols, stream, seed):
    _, s, w = inputs(dev, rows, cols, stream, seed)
    g = gen(dev, seed + 1)
    dy = (torch.randn((rows, cols), generator=g, device=dev) * 1e-2).bfloat16()
    dres = (torch.randn((rows, cols), generator=g, device=dev) * 1e-2).to(s.dtype)
    rstd = torch.cat([torch.rsqrt(p.float().square().mean(1) + 1e-5) for p in s.split(4096)])
    return dy, s, w, rstd, dres


# rows of a team of 1, 4 and 8 waves, more of them than there are teams; one workgroup with 2 to 5 rows
@pytest.mark.parametrize("rows,cols", [(2, 96), (5, 704), (5, 2880), (4, 8224), (3, 20000), (700, 2880), (517, 4096), (1200, 5056), (900, 8192),
                                       (600, 8224), (300, 24576), (2100, 416), (5000, 64), (9001, 800)])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("with_dres", [True, False])
def test_backward_of_several_rows_a_team(dev, rows, cols, stream, with_dres):
    dy, s, w, rstd, dres = gradients(dev, rows, cols, stream, rows + cols)
    dres = dres if with_dres else None
    ds, dw = check_backward(dy, s, w, rstd, dres, stream)
    # each row's gradient is a row of a call of its own
    for r in (0, rows // 2, rows - 1):
        one, _ = backward(dy[r:r + 1], s[r:r + 1], w, rstd[r:r + 1], None if dres is None else dres[r:r + 1], stream)
        assert torch.equal(one[0], ds[r])
    # added to what is there, in place of dres: the same bits, one more addition
    ds2, dw2 = backward(dy, s, w, rstd, dres.clone() if with_dres else None, stream, 1, torch.full_like(dw, 0.5), in_place=with_dres)
    assert torch.equal(ds2, ds)
    assert ((dw2.to(F64) - (dw.to(F64) + 0.5)).abs() <= 2.0 ** -24 * (dw.abs() + 0.5)).all()


# just above 80 MB of traffic, at each kernel's width
LARGE = [(45000, 288), (17000, 672), (5300, 2048), (5300, 2080), (2700, 4096), (1800, 6144), (1350, 8192), (700, 16384), (350, 32768)]


@pytest.mark.parametrize("rows,cols", LARGE)
@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("codes", ["none", "mxfp8", "rows"])
def test_forward_past_the_caches(dev, rows, cols, stream, codes):
    assert rows * cols * (12 if stream == "f32" else 8) > 80 << 20
    x, res, w = inputs(dev, rows, cols, stream, rows + cols)
    got = forward(x, res, w, stream, codes)
    check_forward(x, res, w, stream, codes, got)
    # a third of the rows stays in the caches: the same bits
    n = rows // 3
    assert n * cols * (12 if stream == "f32" else 8) < 80 << 20
    for a in (0, rows - n):
        part = forward(x[a:a + n], res[a:a + n], w, stream, codes)
        assert all(v is None or torch.equal(v, got[k][a:a + n]) for k, v in part.items())


@pytest.mark.parametrize("rows,cols", LARGE)
@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("with_dres", [True, False])
def test_backward_past_the_caches(dev, rows, cols, stream, with_dres):
    assert rows * cols * (14 if stream == "f32" else 8) > 80 << 20
    dy, s, w, rstd, dres = gradients(dev, rows, cols, stream, rows + cols)
    dres = dres if with_dres else None
    ds, _ = check_backward(dy, s, w, rstd, dres, stream)
    n = rows // 3
    assert n * cols * (14 if stream == "f32" else 8) < 80 << 20
    for a in (0, rows - n):
        part, _ = backward(dy[a:a + n], s[a:a + n], w, rstd[a:a + n], None if dres is None else dres[a:a + n], stream)
        assert torch.equal(part, ds[a:a + n])


@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_both_sides_of_the_border(dev, stream):
    """The last call that stays in the caches and the first that does not, of one width: the rows that they share agree."""
    cols = 4096
    for per, both in ((12 if stream == "f32" else 8, "forward"), (14 if stream == "f32" else 8, "backward")):
        rows = (80 << 20) // (cols * per) + 1
        assert (rows - 1) * cols * per <= 80 << 20 < rows * cols * per
        if both == "forward":
            x, res, w = inputs(dev, rows, cols, stream, 3)
            over, under = forward(x, res, w, stream, "mxfp8"), forward(x[1:], res[1:], w, stream, "mxfp8")
            assert all(torch.equal(v, over[k][1:]) for k, v in under.items())
        else:
            dy, s, w, rstd, dres = gradients(dev, rows, cols, stream, 4)
            over, _ = backward(dy, s, w, rstd, dres, stream)
            under, _ = backward(dy[1:], s[1:], w, rstd[1:], dres[1:], stream)
            assert torch.equal(under, over[1:])
