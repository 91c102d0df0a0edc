"""The norm's 8-bit output as the operand of the grouped GEMM: codes and scales
of pt_rmsnorm_fwd, gathered by the router's token_of, go to pt_grouped_gemm_fwd
as they are.

Tolerance, derived: products of codes are exact, K of them are summed in fp32
(K * 2^-24 of the sum of their sizes), the factors' product and its application
round twice, the output once (2^-8).  Against the product of the unrounded norm:
a code is off by 2^-4 of its value or half of the smallest step (2^-10 of its
block's or row's unit); the weights are the codes' values in both.
"""
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.mark.parametrize("T,E,k,K,N", [(50, 8, 2, 256, 128), (300, 12, 4, 416, 96), (7, 5, 3, 2880, 64)])
@pytest.mark.parametrize("kind", ["mxfp8", "rows"])
def test_norm_router_product(dev, T, E, k, K, N, kind):
    g = torch.Generator(device=dev).manual_seed(T + K)
    x, res = (torch.randn((T, K), generator=g, device=dev).bfloat16() for _ in range(2))
    weight = (1 + 0.2 * torch.randn(K, generator=g, device=dev)).bfloat16()
    z = torch.randn((T, E), generator=g, device=dev)
    w = (torch.randn((E, N, K), generator=g, device=dev) * K ** -0.5).bfloat16()
    mx = kind == "mxfp8"
    dtype = ptm.PT_MXFP8_E4M3 if mx else ptm.PT_FP8_E4M3_ROWWISE

    def u8(*shape):
        return torch.empty(shape, dtype=torch.uint8, device=dev)

    def f32(*shape):
        return torch.empty(shape, device=dev)

    h, q, wq = torch.empty_like(x), u8(T, K), u8(E, N, K)
    s, ws = (u8(T, K // 32), u8(E, N, K // 32)) if mx else (f32(T), f32(E, N))
    ptm.pt_rmsnorm_fwd(x, res, weight, h, None, q, s, None, T, K, 1e-5, ptm.PT_BF16, dtype)
    if mx:
        ptm.pt_mx_quantize(w, wq, ws, E * N, K, ptm.PT_MXFP8_E4M3)
    else:
        ptm.pt_fp8_quantize_rows(w, wq, f32(E * N), ws, E * N, K)
    M = T * k
    ids, tw, lens = torch.empty((T, k), dtype=torch.int32, device=dev), f32(T, k), torch.empty(E, dtype=torch.int64, device=dev)
    row_of, token_of = torch.empty((T, k), dtype=torch.int32, device=dev), torch.empty(M, dtype=torch.int32, device=dev)
    ptm.pt_moe_route(z, None, ids, tw, lens, row_of, token_of, T, E, k, workspace=u8(ptm.pt_moe_route_workspace_size(T, E, k)))
    a, sa = q.index_select(0, token_of), s.index_select(0, token_of)
    out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    gws = u8(ptm.pt_grouped_gemm_workspace_size(ptm.PT_OP_FWD, E, M, N, K, dtype))
    gws[:4] = 0
    ptm.pt_grouped_gemm_fwd(a, sa, wq, ws, out, None, lens, None, E, M, N, K, dtype, 1, ptm.PT_EPI_NONE, workspace=gws)
    assert ptm.pt_read_error_flags(gws) == 0

    def value(codes, scales):
        v = codes.cpu().view(torch.float8_e4m3fn).to(F64)
        if mx:
            return v * torch.pow(torch.tensor(2.0, dtype=F64), scales.cpu().to(F64) - 127).repeat_interleave(32, -1)
        return v * scales.cpu().to(F64).unsqueeze(-1)

    av, wv, got = value(a, sa), value(wq, ws), out.cpu().to(F64)
    t = token_of.cpu().long()
    hh = h.cpu().to(F64)
    v = (hh * (hh.square().mean(1, keepdim=True) + 1e-5).pow(-0.5) * weight.cpu().to(F64))[t]
    unit = torch.pow(torch.tensor(2.0, dtype=F64), sa.cpu().to(F64) - 127).repeat_interleave(32, -1) if mx else sa.cpu().to(F64)[:, None]
    off = (2.0 ** -4 + 1e-5) * v.abs() + 2.0 ** -10 * unit
    at = 0
    for e, n in enumerate(lens.tolist()):
        r = slice(at, at + n)
        at += n
        ref, size = av[r] @ wv[e].t(), av[r].abs() @ wv[e].abs().t()
        tol = 2.0 ** -8 * ref.abs() + (K + 4) * 2.0 ** -24 * size
        assert ((got[r] - ref).abs() <= tol).all()
        assert ((got[r] - v[r] @ wv[e].t()).abs() <= tol + (1 + 2.0 ** -8) * (off[r] @ wv[e].abs().t())).all()
    assert at == M
