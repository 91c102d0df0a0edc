"""CPU checks of the dense operators' entry points: what they refuse before any
device call, their workspace sizes, and the header's constants."""
import ctypes
import math
import os
import re

import pytest

from conftest import ROOT

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
FWD, DGRAD, WGRAD = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    import moe_expert_grouped_gemm_amd as pt
    return pt.load(require_gpu=False)


@pytest.fixture(scope="module")
def buf():
    """A 16-byte aligned host address that stands for every operand: no call here gets as far as reading it."""
    raw = ctypes.create_string_buffer(4096)
    p = (ctypes.addressof(raw) + 63) // 64 * 64
    yield p
    del raw


def test_constants_match_the_header():
    import moe_expert_grouped_gemm_amd as pt
    text = open(os.path.join(ROOT, "include", "ptgg.h")).read()
    names = re.findall(r"\b(PT_ACT_\w+|PT_BLOCK_GATE_\w+)\s*=\s*(\d+)", text)
    assert len(names) == 10
    for name, value in names:
        assert getattr(pt, name) == int(value), name


def widths(f):
    """The refusals of sizes that the products share."""
    assert f(M=-1) == INVALID and f(N=0) == INVALID and f(K=0) == INVALID and f(N=-8) == INVALID
    assert f(N=60) == UNSUPPORTED and f(K=36) == UNSUPPORTED
    assert f(M=(1 << 23) + 1) == UNSUPPORTED and f(N=(1 << 17) + 8) == UNSUPPORTED and f(K=(1 << 17) + 8) == UNSUPPORTED
    assert f(M=1 << 23, N=1 << 16) == UNSUPPORTED and f(M=1 << 23, K=1 << 16) == UNSUPPORTED


def test_linear_forward_refusals(L, buf):
    import moe_expert_grouped_gemm_amd as pt
    cut = (100, 264, 4096)
    need = pt.pt_linear_workspace_size(FWD, *cut)
    assert need > 0

    def f(M=4, N=64, K=64, act=0, dt=0, limit=0.0, x=buf, w=buf, bias=buf, res=buf, out=buf, c=buf, ws=buf, n=1 << 40):
        return L.pt_linear_fwd(x, w, bias, res, out, c, M, N, K, act, dt, limit, ws, n, None)
    widths(f)
    assert f(act=-1) == INVALID and f(act=6) == INVALID and f(limit=math.nan) == INVALID
    assert f(dt=1) == UNSUPPORTED and f(dt=4) == UNSUPPORTED and f(act=5, N=72) == UNSUPPORTED
    for name in ("x", "w", "out"):
        assert f(**{name: None}) == INVALID, name
    for name in ("x", "w", "bias", "res", "out", "c"):
        assert f(**{name: buf + 8}) == MISALIGNED, name
    M, N, K = cut
    assert f(M, N, K, ws=None) == WORKSPACE and f(M, N, K, n=need - 1) == WORKSPACE and f(M, N, K, ws=buf + 8) == MISALIGNED
    assert f(M=0, x=None, w=None, out=None) == OK


def test_linear_dgrad_refusals(L, buf):
    import moe_expert_grouped_gemm_amd as pt
    cut = (100, 4096, 264)
    need = pt.pt_linear_workspace_size(DGRAD, *cut)
    assert need > 0

    def f(M=4, N=64, K=64, act=0, limit=0.0, dy=buf, w=buf, c=None, add=buf, dx=buf, ws=buf, n=1 << 40):
        return L.pt_linear_dgrad(dy, w, c, add, dx, M, N, K, act, limit, ws, n, None)
    widths(f)
    assert f(act=6) == INVALID and f(limit=math.nan) == INVALID
    assert f(c=buf) == INVALID and f(act=1) == INVALID                 # saved sums and an activation belong together
    assert f(act=5, c=buf) == INVALID                                  # nothing is added to the gradients of gates and ups
    for name in ("dy", "w", "dx"):
        assert f(**{name: None}) == INVALID, name
    for name in ("dy", "w", "add", "dx"):
        assert f(**{name: buf + 8}) == MISALIGNED, name
    assert f(act=1, c=buf + 8) == MISALIGNED
    M, N, K = cut
    assert f(M, N, K, ws=None) == WORKSPACE and f(M, N, K, n=need - 1) == WORKSPACE and f(M, N, K, ws=buf + 8) == MISALIGNED
    assert f(M=0, dy=None, w=None, dx=None) == OK


def test_linear_wgrad_refusals(L, buf):
    import moe_expert_grouped_gemm_amd as pt
    need = pt.pt_linear_workspace_size(WGRAD, 5000, 64, 264)

    def f(M=5000, N=64, K=264, acc=0, x=buf, dy=buf, dw=buf, db=buf, ws=buf, n=1 << 40):
        return L.pt_linear_wgrad(x, dy, dw, db, M, N, K, acc, ws, n, None)
    widths(f)
    assert f(acc=2) == INVALID and f(acc=-1) == INVALID
    for name in ("x", "dy", "dw"):
        assert f(**{name: None}) == INVALID, name
    for name in ("x", "dy", "dw", "db"):
        assert f(**{name: buf + 8}) == MISALIGNED, name
    assert f(ws=None) == WORKSPACE and f(n=need - 1) == WORKSPACE and f(ws=buf + 8) == MISALIGNED
    assert f(M=0, acc=1, x=None, dy=None, dw=None) == OK
    assert f(M=0, dw=None) == INVALID                                  # zeros have to go somewhere


def test_act_bwd_refusals(L, buf):
    def f(M=4, N=64, act=1, limit=0.0, dout=buf, c=buf, dc=buf):
        return L.pt_linear_act_bwd(dout, c, dc, M, N, act, limit, None)
    assert f(M=-1) == INVALID and f(N=0) == INVALID and f(act=0) == INVALID and f(act=6) == INVALID
    assert f(limit=math.nan) == INVALID and f(N=60) == UNSUPPORTED and f(N=72, act=5) == UNSUPPORTED
    for name in ("dout", "c", "dc"):
        assert f(**{name: None}) == INVALID and f(**{name: buf + 8}) == MISALIGNED, name
    assert f(M=0, dout=None, c=None, dc=None) == OK


def test_block_norm_forward_refusals(L, buf):
    def f(rows=4, cols=64, eps=1e-5, a=1.0, b=1.0, kind=0, stream=0, codes=0, x=buf, res=buf, post=buf, gate=None, pre=buf,
          h=buf, y=buf, q=None, sc=None, r1=buf, r2=buf):
        return L.pt_block_norm_fwd(x, res, post, gate, pre, h, y, q, sc, r1, r2, rows, cols, eps, a, b, kind, stream, codes, None)
    assert f(rows=-1) == INVALID and f(cols=0) == INVALID and f(eps=-1.0) == INVALID and f(eps=math.nan) == INVALID
    assert f(a=math.nan) == INVALID and f(b=math.nan) == INVALID and f(kind=4) == INVALID and f(kind=-1) == INVALID
    assert f(stream=1) == UNSUPPORTED and f(codes=2, q=buf, sc=buf) == UNSUPPORTED
    assert f(cols=60) == UNSUPPORTED and f(cols=72, codes=1, q=buf, sc=buf) == UNSUPPORTED
    assert f(cols=16392) == UNSUPPORTED and f(rows=(1 << 23) + 1) == UNSUPPORTED
    for name in ("x", "res", "h", "y"):
        assert f(**{name: None}) == INVALID, name
    assert f(gate=buf) == INVALID and f(kind=1) == INVALID              # a gate and its kind belong together
    assert f(q=buf) == INVALID and f(codes=1, q=buf) == INVALID and f(codes=4, sc=buf) == INVALID
    assert f(pre=None) == INVALID and f(pre=None, y=None) == INVALID    # outputs of a norm that is not there
    assert f(post=None) == INVALID
    for name in ("x", "res", "post", "pre", "h", "y"):
        assert f(**{name: buf + 8}) == MISALIGNED, name
    assert f(kind=1, gate=buf + 8) == MISALIGNED and f(kind=3, gate=buf + 8) == MISALIGNED and f(kind=2, gate=buf + 2) == MISALIGNED
    assert f(codes=1, q=buf + 4, sc=buf) == MISALIGNED and f(codes=4, q=buf, sc=buf + 2) == MISALIGNED
    assert f(r1=buf + 1) == MISALIGNED and f(r2=buf + 1) == MISALIGNED
    assert f(rows=0, x=None, res=None, h=None, y=None) == OK


def test_block_norm_backward_refusals(L, buf):
    import moe_expert_grouped_gemm_amd as pt
    need = pt.pt_block_norm_workspace_size(100, 64)

    def f(rows=100, cols=64, a=1.0, b=1.0, kind=1, stream=0, acc=0, dy=buf, dres=buf, x=buf, s=buf, post=buf, gate=buf, pre=buf,
          r1=buf, r2=buf, dx=buf, dr=buf, dg=buf, dpost=buf, dpre=buf, ws=buf, n=None):
        return L.pt_block_norm_bwd(dy, dres, x, s, post, gate, pre, r1, r2, dx, dr, dg, dpost, dpre, rows, cols, a, b, kind, stream,
                                   acc, ws, need if n is None else n, None)
    assert f(rows=-1) == INVALID and f(cols=0) == INVALID and f(acc=2) == INVALID and f(kind=4) == INVALID
    assert f(a=math.nan) == INVALID and f(b=math.nan) == INVALID
    assert f(stream=2) == UNSUPPORTED and f(cols=68) == UNSUPPORTED and f(cols=16392) == UNSUPPORTED
    for name in ("dy", "x", "s", "gate", "r1", "r2", "dx", "dr"):
        assert f(**{name: None}) == INVALID, name
    assert f(kind=0, gate=None) == INVALID and f(kind=0, dg=None) == INVALID       # the gradient of no gate; a gate of no kind
    assert f(post=None) == INVALID and f(pre=None, dy=None) == INVALID             # gradients of weights that are not there
    assert f(pre=None, dpre=None) == INVALID                                       # dy without its norm
    assert f(pre=None, dpre=None, dy=None, dres=None) == INVALID
    for name in ("dy", "dres", "x", "s", "post", "gate", "pre", "dx", "dr", "dg", "dpost", "dpre"):
        assert f(**{name: buf + 8}) == MISALIGNED, name
    assert f(kind=2, gate=buf + 2) == MISALIGNED and f(kind=2, dg=buf + 2) == MISALIGNED
    assert f(ws=None) == WORKSPACE and f(n=need - 1) == WORKSPACE and f(ws=buf + 4) == MISALIGNED
    assert f(rows=0, acc=1) == OK and f(rows=0, dg=None, dpost=None, dpre=None) == OK


def test_combine_refusals(L, buf):
    def f(T=4, M=8, H=64, k=2, rows=buf, w=buf, row=buf, base=buf, out=buf):
        return L.pt_moe_combine(rows, w, row, base, out, T, M, H, k, None)

    def b(T=4, M=8, H=64, k=2, dout=buf, rows=buf, w=buf, row=buf, dr=buf, dw=buf):
        return L.pt_moe_combine_bwd(dout, rows, w, row, dr, dw, T, M, H, k, None)
    for g in (f, b):
        assert g(T=-1) == INVALID and g(M=-1) == INVALID and g(H=0) == INVALID and g(k=0) == INVALID
        assert g(H=60) == UNSUPPORTED and g(H=32776) == UNSUPPORTED and g(k=17) == UNSUPPORTED
        assert g(T=(1 << 23) + 1) == UNSUPPORTED and g(M=1 << 31) == UNSUPPORTED
        assert g(rows=None) == INVALID and g(row=None) == INVALID
        assert g(rows=buf + 8) == MISALIGNED and g(w=buf + 2) == MISALIGNED and g(row=buf + 2) == MISALIGNED
    assert f(out=None) == INVALID and f(base=buf + 8) == MISALIGNED and f(out=buf + 8) == MISALIGNED
    assert b(dout=None) == INVALID and b(dr=None, dw=None) == INVALID
    assert b(dout=buf + 8) == MISALIGNED and b(dr=buf + 8) == MISALIGNED and b(dw=buf + 2) == MISALIGNED
    assert f(T=0, rows=None, row=None, out=None) == OK and b(T=0, dout=None, row=None) == OK


def test_workspace_sizes():
    import moe_expert_grouped_gemm_amd as pt
    # sizes and operators that the calls refuse need nothing, no rows neither
    for op in (FWD, DGRAD, WGRAD):
        assert pt.pt_linear_workspace_size(op, -1, 64, 64) == 0 and pt.pt_linear_workspace_size(op, 10, 60, 64) == 0
        assert pt.pt_linear_workspace_size(op, 0, 64, 64) == 0
    assert pt.pt_linear_workspace_size(3, 10, 64, 64) == 0
    # a few rows and products that fill the chip are not cut
    assert pt.pt_linear_workspace_size(FWD, 1, 4096, 4096) == 0 and pt.pt_linear_workspace_size(FWD, 16, 8192, 8192) == 0
    assert pt.pt_linear_workspace_size(FWD, 16384, 8192, 4096) == 0
    # fp32 sums of every part elsewhere: a whole number of products
    n = pt.pt_linear_workspace_size(DGRAD, 100, 4096, 264)
    assert n >= 2 * 100 * 264 * 4
    assert pt.pt_block_norm_workspace_size(0, 64) == 0 and pt.pt_block_norm_workspace_size(10, 16392) == 0
    assert pt.pt_block_norm_workspace_size(1 << 20, 4096) % (2 * 4096 * 4) == 0


def test_binding_refuses_what_the_library_cannot_see():
    """Strided tensors and tensors of the host."""
    import torch

    import moe_expert_grouped_gemm_amd as pt
    if not torch.cuda.is_available():
        with pytest.raises(RuntimeError):
            pt.pt_linear_fwd(None, None, None, None, None, None, 1, 8, 8)
        pytest.skip("no GPU")
    t = torch.zeros((8, 16), device="cuda", dtype=torch.bfloat16)
    for bad in (t[:, :8], t.t(), t.cpu()):
        with pytest.raises(ValueError):
            pt.pt_linear_fwd(bad, t, None, None, t, None, 8, 8, 8)


def test_no_rows_still_need_the_gate(L, buf):
    """The gradients of weights that are written without rows: zeros times the gate, which has to be there."""
    def f(kind, gate, ws=buf):
        return L.pt_block_norm_bwd(None, None, None, None, buf, gate, buf, None, None, None, None, buf if kind else None, buf, buf,
                                   0, 64, 1.0, 1.0, kind, 0, 0, ws, 1 << 20, None)
    assert f(1, None) == INVALID and f(2, None) == INVALID and f(0, buf) == INVALID


def test_most_elements(L, buf):
    rows = 1 << 23
    assert L.pt_block_norm_fwd(buf, buf, None, None, None, buf, None, None, None, None, None, rows, 8200, 1e-5, 1.0, 1.0, 0, 0, 0,
                               None) == UNSUPPORTED
    assert L.pt_moe_combine(buf, None, buf, None, buf, rows, 8, 8200, 1, None) == UNSUPPORTED
    assert L.pt_moe_combine_bwd(buf, buf, None, buf, buf, None, rows, 8, 8200, 1, None) == UNSUPPORTED
