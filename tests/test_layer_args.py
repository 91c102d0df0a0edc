"""CPU checks of the norm, router and few-token entry points: what they refuse
before any device call, their workspace sizes, and the header's constants."""
import ctypes
import math
import os
import re

import pytest

from conftest import ROOT

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4


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
    for name in ("PT_FP32", "PT_GATE_SOFTMAX", "PT_GATE_SIGMOID"):
        assert int(re.search(r"\b%s\s*=\s*(\d+)" % name, text).group(1)) == getattr(pt, name)
    for name in ("PT_MAX_TOPK", "PT_FEW_TOKENS"):
        assert int(re.search(r"#define\s+%s\s+(\d+)" % name, text).group(1)) == getattr(pt, name)


def test_norm_forward_refusals(L, buf):
    def f(rows=4, cols=64, eps=1e-5, stream=0, codes=0, x=buf, res=buf, w=buf, ro=buf, y=buf, q=None, sc=None, rstd=buf):
        return L.pt_rmsnorm_fwd(x, res, w, ro, y, q, sc, rstd, rows, cols, eps, stream, codes, None)
    assert f(rows=-1) == INVALID and f(cols=0) == INVALID
    assert f(eps=-1.0) == INVALID and f(eps=math.nan) == INVALID
    assert f(stream=1) == UNSUPPORTED and f(stream=3) == UNSUPPORTED
    assert f(codes=2, q=buf, sc=buf) == UNSUPPORTED and f(codes=3, q=buf, sc=buf) == UNSUPPORTED
    assert f(cols=60) == UNSUPPORTED
    assert f(cols=72, codes=1, q=buf, sc=buf) == UNSUPPORTED           # whole blocks of 32 only
    assert f(cols=32776) == UNSUPPORTED and f(rows=(1 << 23) + 1) == UNSUPPORTED
    assert f(x=None) == INVALID and f(w=None) == INVALID
    assert f(ro=None) == INVALID                                       # the stream would be lost
    assert f(y=None) == INVALID                                        # no output at all
    assert f(q=buf) == INVALID and f(sc=buf) == INVALID                # codes that were not asked for
    assert f(codes=1, q=buf) == INVALID and f(codes=4, sc=buf) == INVALID
    for name in ("x", "res", "w", "ro", "y"):
        assert f(**{name: buf + 8}) == MISALIGNED, name
    assert f(codes=1, q=buf + 4, sc=buf) == MISALIGNED and f(codes=4, q=buf, sc=buf + 2) == MISALIGNED
    assert f(rstd=buf + 1) == MISALIGNED
    assert f(rows=0, x=None, w=None, ro=None, y=None) == OK


def test_norm_backward_refusals(L, buf):
    import moe_expert_grouped_gemm_amd as pt
    need = pt.pt_rmsnorm_workspace_size(100, 64)

    def f(rows=100, cols=64, stream=0, acc=0, dy=buf, s=buf, w=buf, rstd=buf, dres=buf, ds=buf, dw=buf, ws=buf, n=None):
        return L.pt_rmsnorm_bwd(dy, s, w, rstd, dres, ds, dw, rows, cols, stream, acc, ws, need if n is None else n, None)
    assert f(rows=-1) == INVALID and f(cols=0) == INVALID and f(acc=2) == INVALID
    assert f(stream=2) == UNSUPPORTED and f(cols=68) == UNSUPPORTED and f(cols=40000) == UNSUPPORTED
    for name in ("dy", "s", "w", "rstd", "ds"):
        assert f(**{name: None}) == INVALID, name
    for name in ("dy", "s", "w", "dres", "ds", "dw"):
        assert f(**{name: buf + 4}) == MISALIGNED, name
    assert f(ws=None) == WORKSPACE and f(n=need - 1) == WORKSPACE and f(ws=buf + 4) == MISALIGNED
    assert f(rows=0, acc=1) == OK and f(rows=0, dw=None) == OK


def test_route_refusals(L, buf):
    import moe_expert_grouped_gemm_amd as pt
    need = pt.pt_moe_route_workspace_size(100, 32, 4)

    def f(T=100, E=32, k=4, dt=5, gate=0, renorm=1, scale=1.0, z=buf, bias=None, ids=buf, w=buf, lens=buf, row=buf,
          tok=buf, ws=buf, n=None):
        return L.pt_moe_route(z, bias, ids, w, lens, row, tok, T, E, k, dt, gate, renorm, scale, ws,
                              need if n is None else n, None)
    assert f(T=-1) == INVALID and f(E=0) == INVALID and f(k=0) == INVALID and f(k=33) == INVALID
    assert f(E=1025, k=4) == UNSUPPORTED and f(k=17) == UNSUPPORTED and f(T=(1 << 23) + 1) == UNSUPPORTED
    assert f(gate=2) == INVALID and f(renorm=2) == INVALID and f(scale=math.nan) == INVALID
    assert f(dt=1) == UNSUPPORTED
    assert f(bias=buf) == INVALID                                      # a bias without sigmoid scores
    for name in ("z", "ids", "w", "lens", "row", "tok"):
        assert f(**{name: None}) == INVALID, name
    assert f(z=buf + 4) == MISALIGNED and f(lens=buf + 4) == MISALIGNED and f(row=buf + 2) == MISALIGNED
    assert f(gate=1, bias=buf + 2) == MISALIGNED
    assert f(ws=None, n=0) == WORKSPACE and f(n=need - 1) == WORKSPACE

    def b(T=10, E=32, k=4, dt=5, gate=0, renorm=1, scale=1.0, z=buf, ids=buf, dw=buf, dz=buf):
        return L.pt_moe_route_bwd(z, ids, dw, dz, T, E, k, dt, gate, renorm, scale, None)
    assert b(T=-1) == INVALID and b(k=40) == INVALID and b(E=2000) == UNSUPPORTED and b(dt=4) == UNSUPPORTED
    assert b(gate=-1) == INVALID and b(renorm=-1) == INVALID
    for name in ("z", "ids", "dw", "dz"):
        assert b(**{name: None}) == INVALID, name
    assert b(z=buf + 8) == MISALIGNED and b(dz=buf + 8) == MISALIGNED and b(ids=buf + 1) == MISALIGNED
    assert b(T=0, z=None, ids=None, dw=None, dz=None) == OK


def test_few_tokens_refusals(L, buf):
    import moe_expert_grouped_gemm_amd as pt
    need = pt.pt_moe_few_tokens_workspace_size(8, 16, 64, 96, 4)

    def f(T=8, E=16, H=64, I=96, k=4, dt=5, gate=0, renorm=1, scale=1.0, wt=0, limit=0.0, x=buf, z=buf, bias=None,
          w1=buf, s1=None, w2=buf, s2=None, out=buf, ids=buf, w=buf, ws=buf, n=None):
        return L.pt_moe_few_tokens(x, z, bias, w1, s1, w2, s2, out, ids, w, T, E, H, I, k, dt, gate, renorm, scale, wt,
                                   limit, ws, need if n is None else n, None)
    assert f(T=-1) == INVALID and f(H=0) == INVALID and f(I=0) == INVALID and f(k=17, E=16) == INVALID
    assert f(T=65) == UNSUPPORTED and f(H=68) == UNSUPPORTED and f(I=100) == UNSUPPORTED
    assert f(H=72, wt=1, s1=buf, s2=buf) == UNSUPPORTED and f(I=72, wt=2, s1=buf, s2=buf) == UNSUPPORTED
    assert f(H=16392) == UNSUPPORTED and f(I=16392) == UNSUPPORTED
    assert f(wt=3) == UNSUPPORTED and f(wt=4) == UNSUPPORTED and f(wt=5) == UNSUPPORTED and f(dt=2) == UNSUPPORTED
    assert f(limit=math.nan) == INVALID and f(gate=3) == INVALID and f(bias=buf) == INVALID
    for name in ("x", "z", "w1", "w2", "out", "ids", "w"):
        assert f(**{name: None}) == INVALID, name
    assert f(s1=buf) == INVALID and f(s2=buf) == INVALID               # bf16 weights have no scales
    assert f(wt=1, s1=buf) == INVALID and f(wt=2, s2=buf) == INVALID
    for name in ("x", "z", "w1", "w2", "out", "ws"):
        assert f(**{name: buf + 8}) == MISALIGNED, name
    assert f(ws=None) == WORKSPACE and f(n=need - 1) == WORKSPACE
    assert f(T=0, x=None, z=None, out=None, ws=None) == OK


def test_workspace_sizes():
    import moe_expert_grouped_gemm_amd as pt
    # sizes that the call refuses need nothing
    assert pt.pt_rmsnorm_workspace_size(-1, 64) == 0 and pt.pt_moe_route_workspace_size(10, 4, 5) == 0
    assert pt.pt_moe_few_tokens_workspace_size(65, 8, 64, 64, 2) == 0
    # one part of the weight gradient for few rows, then one fp32 row of it per part
    assert pt.pt_rmsnorm_workspace_size(1, 4096) == 0
    assert pt.pt_rmsnorm_workspace_size(1 << 20, 4096) % (4096 * 4) == 0
    # the router of one chunk of tokens keeps its counts on the chip
    assert pt.pt_moe_route_workspace_size(64, 256, 8) == 256 < pt.pt_moe_route_workspace_size(65, 256, 8)
    # h in bf16 and the experts' outputs in fp32 for every pair, at least
    assert pt.pt_moe_few_tokens_workspace_size(64, 8, 4096, 2048, 4) >= 256 * (2048 * 2 + 4096 * 4)
