"""One MoE block of a transformer on this package: residual RMS norm, router,
experts, a shared expert, and the norms between this block and the next -- a
training step with its backward, and decoding.

    python examples/moe_block.py            # 4096 tokens of 1024, 32 experts of inner size 512, 4 each, a shared one of 1024

Every product, norm, choice and join of rows is the package's; torch holds the
memory, adds up the experts' row counts, lays the router's gradient out, and
projects the router where the experts are no multiple of 8.
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_grouped_gemm_amd as pt  # noqa: E402

EPS = 1e-5


class MoeBlock:
    """Weights in bf16 with fp32 gradients; the residual stream in bf16.

    shared: inner size of an expert that every token takes beside its own, or 0.
    close and close_backward put the block's output behind a norm of its own and
    a factor per channel onto the stream, and norm that for the next block."""

    def __init__(self, hidden, inner, experts, topk, device, seed=0, shared=0):
        self.H, self.I, self.E, self.k, self.S = hidden, inner, experts, topk, shared
        self.device = torch.device(device)
        g = torch.Generator(device=self.device).manual_seed(seed)

        def w(*shape):
            return (torch.randn(shape, generator=g, device=self.device) * shape[-1] ** -0.5).bfloat16()

        self.norm = torch.ones(hidden, dtype=torch.bfloat16, device=self.device)
        self.router = w(experts, hidden)
        self.w1, self.w2 = w(experts, 2 * inner, hidden), w(experts, hidden, inner)      # [experts, out, in]
        names = ["norm", "router", "w1", "w2", "post", "gate", "next"]
        if shared:
            self.s1, self.s2 = w(2 * shared, hidden), w(hidden, shared)
            names += ["s1", "s2"]
        self.post, self.next = torch.ones_like(self.norm), torch.ones_like(self.norm)
        self.gate = torch.full_like(self.norm, 0.5)
        self.grad = {n: torch.zeros(getattr(self, n).shape, device=self.device) for n in names}

    def _new(self, shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def _gemm_workspace(self, op, rows, N, K):
        n = pt.pt_grouped_gemm_workspace_size(op, self.E, rows, N, K, pt.PT_BF16)
        return self._new(n, torch.uint8)

    def _linear(self, x, w, out, c=None, residual=None, act=pt.PT_ACT_NONE):
        """out = act(x w^T) + residual; the sums before act into c."""
        M, (N, K) = x.shape[0], w.shape
        pt.pt_linear_fwd(x, w, None, residual, out, c, M, N, K, act,
                         pt.PT_FP32 if out.dtype == torch.float32 else pt.PT_BF16,
                         workspace=self._new(pt.pt_linear_workspace_size(pt.PT_OP_FWD, M, N, K), torch.uint8))
        return out

    def _linear_dgrad(self, dy, w, dx, c=None, add=None, act=pt.PT_ACT_NONE):
        M, (N, K) = dy.shape[0], w.shape
        pt.pt_linear_dgrad(dy, w, c, add, dx, M, N, K, act,
                           workspace=self._new(pt.pt_linear_workspace_size(pt.PT_OP_DGRAD, M, N, K), torch.uint8))
        return dx

    def _linear_wgrad(self, x, dy, grad):
        M, (N, K) = x.shape[0], grad.shape
        pt.pt_linear_wgrad(x, dy, grad, None, M, N, K, 1,
                           workspace=self._new(pt.pt_linear_workspace_size(pt.PT_OP_WGRAD, M, N, K), torch.uint8))

    def _in_parts(self, x):
        """fp32 [T, n] for the products, which take bf16: three parts beside each other whose sum is x to its last bit (8 bits
        each), then zeros up to a multiple of 8 columns."""
        T, n = x.shape
        parts = self._new((T, -(-3 * n // 8) * 8))
        parts[:, 3 * n :] = 0
        for i in range(3):
            part = parts[:, i * n : (i + 1) * n].copy_(x)
            x = x - part.float()
        return parts

    def _norm(self, x, residual, rstd=None):
        stream, y = self._new(x.shape), self._new(x.shape)
        pt.pt_rmsnorm_fwd(x, residual, self.norm, stream, y, None, None, rstd, x.shape[0], self.H, EPS)
        return stream, y

    def _logits(self, y):
        if self.E % 8:      # the products' sizes are multiples of 8
            return (y @ self.router.t()).float()
        return self._linear(y, self.router, self._new((y.shape[0], self.E), torch.float32))

    def _shared(self, y, residual=None, save=True):
        """The shared expert's output, and what its backward needs (save: the sums before SwiGLU too)."""
        c, h = self._new((y.shape[0], 2 * self.S)) if save else None, self._new((y.shape[0], self.S))
        self._linear(y, self.s1, h, c, act=pt.PT_ACT_SWIGLU)
        return self._linear(h, self.s2, self._new(y.shape), residual=residual), c, h

    def forward(self, x, residual):
        """The block's output and the residual stream; what the backward needs stays in self.saved."""
        T, k, E, H, I = x.shape[0], self.k, self.E, self.H, self.I
        rstd = self._new(T, torch.float32)
        stream, y = self._norm(x, residual, rstd)
        logits = self._logits(y)
        ids, weights = self._new((T, k), torch.int32), self._new((T, k), torch.float32)
        lens, row_of = self._new(E, torch.int64), self._new((T, k), torch.int32)
        token_of = self._new(T * k, torch.int32)
        pt.pt_moe_route(logits, None, ids, weights, lens, row_of, token_of, T, E, k, pt.PT_FP32, pt.PT_GATE_SOFTMAX, 1,
                        workspace=self._new(pt.pt_moe_route_workspace_size(T, E, k), torch.uint8))
        M = T * k
        # a token without experts (one that holds a NaN) has -1 in row_of, which the joins skip, and leaves the last rows to
        # nobody: offs keeps the products to the rows that experts have
        offs = torch.zeros(E + 1, dtype=torch.int64, device=self.device)
        torch.cumsum(lens, 0, out=offs[1:])
        a, c, h, o = self._new((M, H)), self._new((M, 2 * I)), self._new((M, I)), self._new((M, H))
        pt.pt_moe_combine_bwd(y, None, None, row_of, a, None, T, M, H, k)       # a[row_of[t, j]] = y[t]
        pt.pt_grouped_gemm_fwd_swiglu_save(a, None, self.w1, None, h, c, lens, offs, E, M, 2 * I, H, pt.PT_BF16, 1,
                                           workspace=self._gemm_workspace(pt.PT_OP_FWD, M, 2 * I, H))
        pt.pt_grouped_gemm_fwd(h, None, self.w2, None, o, None, lens, offs, E, M, H, I, pt.PT_BF16, 1, pt.PT_EPI_NONE,
                               workspace=self._gemm_workspace(pt.PT_OP_FWD, M, H, I))
        base, sc, sh = self._shared(y) if self.S else (None, None, None)
        out = self._new((T, H))
        pt.pt_moe_combine(o, weights, row_of, base, out, T, M, H, k)
        self.saved = (stream, y, rstd, logits, ids, weights, lens, row_of, offs, a, c, h, o, sc, sh)
        return out, stream

    def backward(self, dout, dstream):
        """The gradient of the block's inputs (x and the residual alike); the weights' gradients are added to self.grad.
        dstream: the gradient that reaches the residual stream past this block."""
        stream, y, rstd, logits, ids, weights, lens, row_of, offs, a, c, h, o, sc, sh = self.saved
        T, k, E, H, I = y.shape[0], self.k, self.E, self.H, self.I
        M = T * k
        do, dweights = self._new((M, H)), self._new((T, k), torch.float32)
        pt.pt_moe_combine_bwd(dout, o, weights, row_of, do, dweights, T, M, H, k)
        dc, da = self._new((M, 2 * I)), self._new((M, H))
        pt.pt_grouped_gemm_dgrad_swiglu(do, self.w2, c, dc, lens, offs, E, M, H, I, 1,
                                        workspace=self._gemm_workspace(pt.PT_OP_DGRAD, M, H, I))
        pt.pt_grouped_gemm_wgrad(h, None, do, None, self.grad["w2"], lens, offs, E, M, H, I, pt.PT_BF16, 1, 1,
                                 workspace=self._gemm_workspace(pt.PT_OP_WGRAD, M, H, I))
        pt.pt_grouped_gemm_dgrad(dc, None, self.w1, None, da, lens, offs, E, M, 2 * I, H, pt.PT_BF16, 1,
                                 workspace=self._gemm_workspace(pt.PT_OP_DGRAD, M, 2 * I, H))
        pt.pt_grouped_gemm_wgrad(a, None, dc, None, self.grad["w1"], lens, offs, E, M, 2 * I, H, pt.PT_BF16, 1, 1,
                                 workspace=self._gemm_workspace(pt.PT_OP_WGRAD, M, 2 * I, H))
        dy = self._new((T, H))
        pt.pt_moe_combine(da, None, row_of, None, dy, T, M, H, k)
        dlogits = torch.empty_like(logits)
        pt.pt_moe_route_bwd(logits, ids, dweights, dlogits, T, E, k, pt.PT_FP32, pt.PT_GATE_SOFTMAX, 1)
        d = self._in_parts(dlogits)
        dw = torch.zeros((d.shape[1], H), device=self.device)
        self._linear_wgrad(y, d, dw)
        self.grad["router"] += dw[2 * E : 3 * E] + dw[E : 2 * E] + dw[:E]
        w = [self.router] * 3 + [self.router.new_zeros(d.shape[1] - 3 * E, H)]
        if self.S:
            dsc = self._linear_dgrad(dout, self.s2, self._new((T, 2 * self.S)), sc, act=pt.PT_ACT_SWIGLU)
            self._linear_wgrad(sh, dout, self.grad["s2"])
            self._linear_wgrad(y, dsc, self.grad["s1"])
            d, w = torch.cat((d, dsc), 1), w + [self.s1]
        # through router and shared expert in one product, onto the experts' sum: dy is rounded there and here
        self._linear_dgrad(d, torch.cat(w), dy, add=dy)
        ds = self._new((T, H))
        pt.pt_rmsnorm_bwd(dy, stream, self.norm, rstd, dstream, ds, self.grad["norm"], T, H, pt.PT_BF16, 1,
                          workspace=self._new(pt.pt_rmsnorm_workspace_size(T, H), torch.uint8))
        return ds

    def close(self, out, stream):
        """The stream behind the block, stream + gate * norm(out), and its norm, which the next block reads."""
        T, H = out.shape
        after, y = self._new((T, H)), self._new((T, H))
        rstd = self._new((2, T), torch.float32)
        pt.pt_block_norm_fwd(out, stream, self.post, self.gate, self.next, after, y, None, None, rstd[0], rstd[1], T, H, EPS,
                             gate_kind=pt.PT_BLOCK_GATE_COLS)
        self.closed = (out, after, rstd)
        return after, y

    def close_backward(self, dy, dafter):
        """The gradients of out and stream, of what reaches the next block's norm and the stream past it."""
        out, after, rstd = self.closed
        T, H = out.shape
        dout, dstream = self._new((T, H)), self._new((T, H))
        pt.pt_block_norm_bwd(dy, dafter, out, after, self.post, self.gate, self.next, rstd[0], rstd[1], dout, dstream,
                             self.grad["gate"], self.grad["post"], self.grad["next"], T, H,
                             gate_kind=pt.PT_BLOCK_GATE_COLS, accumulate=1,
                             workspace=self._new(pt.pt_block_norm_workspace_size(T, H), torch.uint8))
        return dout, dstream

    def decode(self, x, residual):
        """The same output for at most 64 tokens: the norm and one call for the whole layer."""
        T = x.shape[0]
        stream, y = self._norm(x, residual)
        logits = self._logits(y)
        out, ids = self._new((T, self.H)), self._new((T, self.k), torch.int32)
        n = pt.pt_moe_few_tokens_workspace_size(T, self.E, self.H, self.I, self.k)
        pt.pt_moe_few_tokens(y, logits, None, self.w1, None, self.w2, None, out, ids, self._new((T, self.k), torch.float32),
                             T, self.E, self.H, self.I, self.k, pt.PT_FP32, pt.PT_GATE_SOFTMAX, 1, 1.0, pt.PT_BF16,
                             workspace=self._new(n, torch.uint8))
        if self.S:
            out, _, _ = self._shared(y, residual=out, save=False)
        return out, stream


def main():
    dev = torch.device("cuda", 0)
    block = MoeBlock(1024, 512, 32, 4, dev, shared=1024)
    g = torch.Generator(device=dev).manual_seed(1)
    x, residual, dout = (torch.randn((4096, 1024), generator=g, device=dev).bfloat16() for _ in range(3))

    def step():
        block.close(*block.forward(x, residual))
        return block.backward(*block.close_backward(dout, dout))

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
