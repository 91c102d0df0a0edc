"""One MoE block of a transformer on this package: residual RMS norm, router,
experts -- a training step with its backward, and decoding.

    python examples/moe_block.py            # 4096 tokens of 1024, 32 experts of inner size 512, 4 each

The norm, the router, the grouped GEMMs and the layer for a few tokens are the
package's; the router's small projection, the gather of the experts' rows and
the weighted sum over a token's slots are torch's.
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_grouped_gemm_amd as pt  # noqa: E402

EPS = 1e-5


class MoeBlock:
    """Weights in bf16 with fp32 gradients; the residual stream in bf16."""

    def __init__(self, hidden, inner, experts, topk, device, seed=0):
        self.H, self.I, self.E, self.k = hidden, inner, experts, topk
        self.device = torch.device(device)
        g = torch.Generator(device=self.device).manual_seed(seed)

        def w(*shape):
            return (torch.randn(shape, generator=g, device=self.device) * shape[-1] ** -0.5).bfloat16()

        self.norm = torch.ones(hidden, dtype=torch.bfloat16, device=self.device)
        self.router = w(experts, hidden)
        self.w1, self.w2 = w(experts, 2 * inner, hidden), w(experts, hidden, inner)      # [experts, out, in]
        self.grad = {n: torch.zeros(getattr(self, n).shape, device=self.device) for n in ("norm", "router", "w1", "w2")}

    def _new(self, shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def _rows(self, n):
        """n rows for a product to fill and a zero one."""
        rows = self._new((n + 1, self.H))
        rows[n].zero_()
        return rows

    def _gemm_workspace(self, op, rows, N, K):
        n = pt.pt_grouped_gemm_workspace_size(op, self.E, rows, N, K, pt.PT_BF16)
        return self._new(n, torch.uint8)

    def _norm(self, x, residual, rstd=None):
        stream, y = self._new(x.shape), self._new(x.shape)
        pt.pt_rmsnorm_fwd(x, residual, self.norm, stream, y, None, None, rstd, x.shape[0], self.H, EPS)
        return stream, y

    def forward(self, x, residual):
        """The block's output and the residual stream; what the backward needs stays in self.saved."""
        T, k, E, H, I = x.shape[0], self.k, self.E, self.H, self.I
        rstd = self._new(T, torch.float32)
        stream, y = self._norm(x, residual, rstd)
        logits = (y @ self.router.t()).float()
        ids, weights = self._new((T, k), torch.int32), self._new((T, k), torch.float32)
        lens, row_of = self._new(E, torch.int64), self._new((T, k), torch.int32)
        token_of = self._new(T * k, torch.int32)
        pt.pt_moe_route(logits, None, ids, weights, lens, row_of, token_of, T, E, k, pt.PT_FP32, pt.PT_GATE_SOFTMAX, 1,
                        workspace=self._new(pt.pt_moe_route_workspace_size(T, E, k), torch.uint8))
        M = T * k
        # a token without experts (one that holds a NaN) has -1 in row_of and leaves the last rows to nobody: it reads row M,
        # which is zero, and offs keeps the products to the rows that experts have
        offs = torch.zeros(E + 1, dtype=torch.int64, device=self.device)
        torch.cumsum(lens, 0, out=offs[1:])
        row_of = torch.where(row_of < 0, M, row_of).long()
        token_of.clamp_(min=0)
        a = y.index_select(0, token_of)
        c, h, o = self._new((M, 2 * I)), self._new((M, I)), self._rows(M)
        pt.pt_grouped_gemm_fwd_swiglu_save(a, None, self.w1, None, h, c, lens, offs, E, M, 2 * I, H, pt.PT_BF16, 1,
                                           workspace=self._gemm_workspace(pt.PT_OP_FWD, M, 2 * I, H))
        pt.pt_grouped_gemm_fwd(h, None, self.w2, None, o, None, lens, offs, E, M, H, I, pt.PT_BF16, 1, pt.PT_EPI_NONE,
                               workspace=self._gemm_workspace(pt.PT_OP_FWD, M, H, I))
        out = (o[row_of].float() * weights.unsqueeze(2)).sum(1).bfloat16()
        self.saved = (stream, y, rstd, logits, ids, weights, lens, row_of, token_of, a, c, h, o, offs)
        return out, stream

    def backward(self, dout, dstream):
        """The gradient of the block's inputs (x and the residual alike); the weights' gradients are added to self.grad.
        dstream: the gradient that reaches the residual stream past this block."""
        stream, y, rstd, logits, ids, weights, lens, row_of, token_of, a, c, h, o, offs = self.saved
        T, k, E, H, I = y.shape[0], self.k, self.E, self.H, self.I
        M = T * k
        dweights = torch.stack([(o[row_of[:, j]].float() * dout.float()).sum(1) for j in range(k)], 1)
        row_weight = torch.zeros(M + 1, device=self.device)
        row_weight[row_of.flatten()] = weights.flatten()
        do = (dout.index_select(0, token_of).float() * row_weight[:M].unsqueeze(1)).bfloat16()
        dc, da = self._new((M, 2 * I)), self._rows(M)
        pt.pt_grouped_gemm_dgrad_swiglu(do, self.w2, c, dc, lens, offs, E, M, H, I, 1,
                                        workspace=self._gemm_workspace(pt.PT_OP_DGRAD, M, H, I))
        pt.pt_grouped_gemm_wgrad(h, None, do, None, self.grad["w2"], lens, offs, E, M, H, I, pt.PT_BF16, 1, 1,
                                 workspace=self._gemm_workspace(pt.PT_OP_WGRAD, M, H, I))
        pt.pt_grouped_gemm_dgrad(dc, None, self.w1, None, da, lens, offs, E, M, 2 * I, H, pt.PT_BF16, 1,
                                 workspace=self._gemm_workspace(pt.PT_OP_DGRAD, M, 2 * I, H))
        pt.pt_grouped_gemm_wgrad(a, None, dc, None, self.grad["w1"], lens, offs, E, M, 2 * I, H, pt.PT_BF16, 1, 1,
                                 workspace=self._gemm_workspace(pt.PT_OP_WGRAD, M, 2 * I, H))
        dlogits = torch.empty_like(logits)
        pt.pt_moe_route_bwd(logits, ids, dweights, dlogits, T, E, k, pt.PT_FP32, pt.PT_GATE_SOFTMAX, 1)
        self.grad["router"] += dlogits.t() @ y.float()
        dy = (da[row_of].float().sum(1) + dlogits @ self.router.float()).bfloat16()
        ds = self._new((T, H))
        pt.pt_rmsnorm_bwd(dy, stream, self.norm, rstd, dstream, ds, self.grad["norm"], T, H, pt.PT_BF16, 1,
                          workspace=self._new(pt.pt_rmsnorm_workspace_size(T, H), torch.uint8))
        return ds

    def decode(self, x, residual):
        """The same output for at most 64 tokens: the norm and one call for the whole layer."""
        T = x.shape[0]
        stream, y = self._norm(x, residual)
        logits = (y @ self.router.t()).float()
        out, ids = self._new((T, self.H)), self._new((T, self.k), torch.int32)
        n = pt.pt_moe_few_tokens_workspace_size(T, self.E, self.H, self.I, self.k)
        pt.pt_moe_few_tokens(y, logits, None, self.w1, None, self.w2, None, out, ids, self._new((T, self.k), torch.float32),
                             T, self.E, self.H, self.I, self.k, pt.PT_FP32, pt.PT_GATE_SOFTMAX, 1, 1.0, pt.PT_BF16,
                             workspace=self._new(n, torch.uint8))
        return out, stream


def main():
    dev = torch.device("cuda", 0)
    block = MoeBlock(1024, 512, 32, 4, dev)
    g = torch.Generator(device=dev).manual_seed(1)
    x, residual, dout = (torch.randn((4096, 1024), generator=g, device=dev).bfloat16() for _ in range(3))

    def step():
        block.forward(x, residual)
        return block.backward(dout, dout)

    for name, run in (("training step, 4096 tokens", step), ("decoding, 8 tokens", lambda: block.decode(x[:8], residual[:8]))):
        for _ in range(5):
            run()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(20):
            run()
        torch.cuda.synchronize()
        print(f"{name}: {(time.perf_counter() - t) / 20 * 1e6:.0f} us")
    out, _ = block.forward(x, residual)
    few, _ = block.decode(x[:8], residual[:8])
    diff = (few.float() - out[:8].float()).norm() / out[:8].float().norm()
    print(f"decoded tokens against the training forward: {diff.item():.1e} of their norm")


if __name__ == "__main__":
    main()
