"""Cases for the dense operators of an MoE block: the matrix product with bias,
activation and residual in its epilogue (forward, data and weight gradient), the
norms after and before a block with its gate and residual scale (forward and
backward), and the weighted sum that brings the experts' rows back to their
tokens (forward and backward).

Shapes follow the package's workloads: hidden size 4096 with experts of inner
size 2048, six per token, and hidden and inner size 2880 with 32 experts, four
per token; 8192 and 16384 tokens for training, a few to tens for serving.
"""
import math

import torch

own = False

EPS = 1e-5
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def listed():
    return [
        # one decoded token through the attention's output projection, added to the residual stream
        {"name": "linear_1", "op": "linear", "rows": 1, "out": 4096, "in": 4096, "act": "none", "bias": False,
         "residual": True, "save": False, "stream": "bf16"},
        # a decode batch of odd size through a shared expert's gate and up projection
        {"name": "linear_45_swiglu", "op": "linear", "rows": 45, "out": 4096, "in": 4096, "act": "swiglu", "bias": False,
         "residual": False, "save": False, "stream": "bf16"},
        # a training batch's router logits: 32 experts, biased, kept in fp32
        {"name": "linear_16384_router", "op": "linear", "rows": 16384, "out": 32, "in": 2880, "act": "none", "bias": True,
         "residual": False, "save": False, "stream": "f32"},
        # a ragged prompt through a biased projection onto an fp32 residual stream
        {"name": "linear_1021_gelu_f32", "op": "linear", "rows": 1021, "out": 2880, "in": 2880, "act": "gelu_tanh",
         "bias": True, "residual": True, "save": False, "stream": "f32"},
        # the training forward of a dense block's FC1, which keeps its output for the backward
        {"name": "linear_8192_swiglu_save", "op": "linear", "rows": 8192, "out": 8192, "in": 4096, "act": "swiglu",
         "bias": False, "residual": False, "save": True, "stream": "bf16"},
        # its FC2's data gradient, which ends in the gradient of FC1's output
        {"name": "linear_dgrad_8192_swiglu", "op": "linear_dgrad", "rows": 8192, "out": 4096, "in": 2048, "act": "swiglu",
         "add": False},
        # the weight and bias gradient of a biased projection
        {"name": "linear_wgrad_16384", "op": "linear_wgrad", "rows": 16384, "out": 2880, "in": 2880, "bias": True},
        # a few decoded tokens between two blocks: the next product takes 8-bit codes
        {"name": "block_norm_5_mxfp8", "op": "block_norm", "rows": 5, "cols": 4096, "stream": "bf16", "gate": "cols",
         "codes": "mxfp8"},
        # a training batch with a gate per element and the residual stream in fp32
        {"name": "block_norm_8192_f32", "op": "block_norm", "rows": 8192, "cols": 4096, "stream": "f32", "gate": "full",
         "codes": "none"},
        # the training step's backward over 16384 tokens, a gate per channel
        {"name": "block_norm_bwd_16384", "op": "block_norm_bwd", "rows": 16384, "cols": 2880, "stream": "bf16",
         "gate": "cols"},
        # the experts' rows of a training batch back to their tokens, on top of a shared expert's output
        {"name": "combine_16384", "op": "combine", "rows": 16384, "cols": 2880, "k": 4, "weights": True, "base": True},
        # the gradients of the experts' rows and of the router's weights, an odd micro-batch
        {"name": "combine_bwd_8191", "op": "combine_bwd", "rows": 8191, "cols": 4096, "k": 6},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _odd(rng, unit, lo, hi):
    """An odd multiple of `unit`: rows of it start at every place of a cache line."""
    return unit * (_log_uniform(rng, lo, hi) | 1)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "linear_dgrad", "linear_wgrad", "block_norm", "block_norm_bwd",
                     "combine", "combine_bwd"])
    rows = _log_uniform(rng, 1, 8192 if op.startswith("linear") else 16384)
    if op.startswith("linear"):
        c = {"op": op, "rows": rows, "out": _odd(rng, 8, 4, 510), "in": _odd(rng, 8, 16, 510)}
        if op == "linear_wgrad":
            return dict(c, bias=rng.random() < 0.5)
        c["act"] = rng.choice(["none", "none", "swiglu", "silu", "relu2", "gelu", "gelu_tanh"])
        if op == "linear_dgrad":
            return dict(c, add=c["act"] == "none" and rng.random() < 0.5)
        if c["act"] == "swiglu":
            c["out"] *= 2
        return dict(c, bias=rng.random() < 0.5, residual=rng.random() < 0.5, save=rng.random() < 0.3,
                    stream=rng.choice(["bf16", "f32"]))
    cols = _odd(rng, 32, 8, 158)
    if op.startswith("block_norm"):
        c = {"op": op, "rows": rows, "cols": cols, "stream": rng.choice(["bf16", "f32"]),
             "gate": rng.choice(["none", "cols", "rows", "full"])}
        if op == "block_norm":
            c["codes"] = rng.choice(["none", "mxfp8", "fp8rows"])
        return c
    c = {"op": op, "rows": rows, "cols": cols, "k": rng.randint(1, 8)}
    if op == "combine":
        c.update(weights=rng.random() < 0.7, base=rng.random() < 0.5)
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda" if torch.cuda.is_available() else "cpu")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=g.device).mul_(std)


def _type(case):
    return F32 if case["stream"] == "f32" else BF16


def _glu(case):
    return 2 if case["act"] == "swiglu" else 1


def _routing(g, T, k):
    """[T, k] rows in expert order, each used once; a few slots have none (-1)."""
    E = 32
    ids = torch.rand((T, E), generator=g, device=g.device).argsort(dim=1)[:, :k]
    if T > 1:
        ids[:, k - 1] = torch.where(torch.rand(T, generator=g, device=g.device) < 0.01, E, ids[:, k - 1])
    order = torch.argsort(ids.flatten(), stable=True)
    row_of = torch.empty_like(order)
    row_of[order] = torch.arange(T * k, device=g.device)
    return torch.where(ids == E, -1, row_of.view(T, k)).int().contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op.startswith("linear"):
        M, N, K = case["rows"], case["out"], case["in"]
        if op == "linear":
            s["x"] = _randn(g, M, K).to(BF16)
            s["w"] = _randn(g, N, K, std=K ** -0.5).to(BF16)
            s["bias"] = _randn(g, N, std=0.3).to(BF16) if case["bias"] else None
            s["residual"] = _randn(g, M, N // _glu(case), std=3.0).to(_type(case)) if case["residual"] else None
        elif op == "linear_dgrad":
            s["dy"] = _randn(g, M, N, std=1e-2).to(BF16)
            s["w"] = _randn(g, N, K, std=K ** -0.5).to(BF16)
            s["c"] = _randn(g, M, K * _glu(case)).to(BF16) if case["act"] != "none" else None
            s["add"] = _randn(g, M, K, std=1e-2).to(BF16) if case["add"] else None
        else:
            s["x"] = _randn(g, M, K).to(BF16)
            s["dy"] = _randn(g, M, N, std=1e-2).to(BF16)
    elif op.startswith("block_norm"):
        R, C, dt = case["rows"], case["cols"], _type(case)
        s["x"] = _randn(g, R, C).mul_(1 + _randn(g, C).abs_()).to(BF16)
        s["post"] = (1 + _randn(g, C, std=0.2)).to(BF16)
        s["pre"] = (1 + _randn(g, C, std=0.2)).to(BF16)
        kind = case["gate"]
        s["gate"] = {"none": lambda: None, "cols": lambda: (0.5 + _randn(g, C, std=0.2)).to(BF16),
                     "rows": lambda: torch.sigmoid(_randn(g, R)),
                     "full": lambda: torch.sigmoid(_randn(g, R, C)).to(BF16)}[kind]()
        s["branch_scale"], s["residual_scale"] = 0.75, 1.25
        if op == "block_norm":
            s["residual"] = _randn(g, R, C, std=3.0).to(dt)
        else:
            s["s"] = _randn(g, R, C, std=3.0).to(dt)
            s["rstd_post"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["rstd_pre"] = torch.rsqrt(s["s"].float().square().mean(1) + EPS)
            s["dy"] = _randn(g, R, C, std=1e-2).to(BF16)
            s["dres"] = _randn(g, R, C, std=1e-2).to(dt)
    else:
        T, H, k = case["rows"], case["cols"], case["k"]
        s["row_of"] = _routing(g, T, k)
        s["y"] = _randn(g, T * k, H).to(BF16)
        s["weights"] = torch.softmax(_randn(g, T, k), 1) if case.get("weights", True) else None
        if op == "combine":
            s["base"] = _randn(g, T, H).to(BF16) if case["base"] else None
        else:
            s["dout"] = _randn(g, T, H, std=1e-2).to(BF16)
    if own:
        _buffers(s, case, g.device)
    return s


def _buffers(s, case, dev):
    """The outputs and the workspace that a program on the package's caller-owned buffers keeps."""
    import moe_expert_grouped_gemm_amd as pt

    def new(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=dev)

    op = case["op"]
    if op.startswith("linear"):
        M, N, K = case["rows"], case["out"], case["in"]
        kind = {"linear": pt.PT_OP_FWD, "linear_dgrad": pt.PT_OP_DGRAD, "linear_wgrad": pt.PT_OP_WGRAD}[op]
        s["workspace"] = new(pt.pt_linear_workspace_size(kind, M, N, K), torch.uint8)
        if op == "linear":
            s["o"] = new((M, N // _glu(case)), _type(case))
            s["c"] = new((M, N), BF16) if case["save"] else None
        elif op == "linear_dgrad":
            s["dx"] = new((M, K * _glu(case)), BF16)
        else:
            s["dw"] = new((N, K), F32)
            s["dbias"] = new(N, F32) if case["bias"] else None
    elif op == "block_norm":
        R, C = case["rows"], case["cols"]
        s["h"], s["o"] = new((R, C), _type(case)), new((R, C), BF16)
        s["rstd_post"], s["rstd_pre"] = new(R, F32), new(R, F32)
        s["q"] = new((R, C), torch.uint8) if case["codes"] != "none" else None
        s["scales"] = {"none": None, "mxfp8": new((R, C // 32), torch.uint8), "fp8rows": new(R, F32)}[case["codes"]]
    elif op == "block_norm_bwd":
        R, C = case["rows"], case["cols"]
        s["dx"], s["dresidual"] = new((R, C), BF16), new((R, C), _type(case))
        s["dpost"], s["dpre"] = new(C, F32), new(C, F32)
        s["dgate"] = {"none": None, "cols": new(C, F32), "rows": new(R, F32), "full": new((R, C), BF16)}[case["gate"]]
        s["workspace"] = new(pt.pt_block_norm_workspace_size(R, C), torch.uint8)
    elif op == "combine":
        s["o"] = new((case["rows"], case["cols"]), BF16)
    else:
        # rows that no slot names are left as they are
        s["drows"] = torch.zeros((case["rows"] * case["k"], case["cols"]), dtype=BF16, device=dev)
        s["dweights"] = new((case["rows"], case["k"]), F32)


# ------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import moe_expert_grouped_gemm_amd as pt
    c = s["case"]
    op = c["op"]
    stream = {"bf16": pt.PT_BF16, "f32": pt.PT_FP32}
    if op.startswith("linear"):
        act = {"none": pt.PT_ACT_NONE, "swiglu": pt.PT_ACT_SWIGLU, "silu": pt.PT_ACT_SILU, "relu2": pt.PT_ACT_RELU2,
               "gelu": pt.PT_ACT_GELU, "gelu_tanh": pt.PT_ACT_GELU_TANH}[c.get("act", "none")]
        M, N, K = c["rows"], c["out"], c["in"]
        if op == "linear":
            pt.pt_linear_fwd(s["x"], s["w"], s["bias"], s["residual"], s["o"], s["c"], M, N, K, act, stream[c["stream"]],
                             workspace=s["workspace"])
            return {"out": s["o"], "c": s["c"]} if c["save"] else {"out": s["o"]}
        if op == "linear_dgrad":
            pt.pt_linear_dgrad(s["dy"], s["w"], s["c"], s["add"], s["dx"], M, N, K, act, workspace=s["workspace"])
            return {"dx": s["dx"]}
        pt.pt_linear_wgrad(s["x"], s["dy"], s["dw"], s["dbias"], M, N, K, 0, workspace=s["workspace"])
        return {"dw": s["dw"], "dbias": s["dbias"]} if c["bias"] else {"dw": s["dw"]}
    if op.startswith("block_norm"):
        gate = {"none": pt.PT_BLOCK_GATE_NONE, "cols": pt.PT_BLOCK_GATE_COLS, "rows": pt.PT_BLOCK_GATE_ROWS,
                "full": pt.PT_BLOCK_GATE_FULL}[c["gate"]]
        R, C = c["rows"], c["cols"]
        if op == "block_norm":
            codes = {"none": pt.PT_BF16, "mxfp8": pt.PT_MXFP8_E4M3, "fp8rows": pt.PT_FP8_E4M3_ROWWISE}[c["codes"]]
            pt.pt_block_norm_fwd(s["x"], s["residual"], s["post"], s["gate"], s["pre"], s["h"], s["o"], s["q"], s["scales"],
                                 s["rstd_post"], s["rstd_pre"], R, C, EPS, s["branch_scale"], s["residual_scale"], gate,
                                 stream[c["stream"]], codes)
            return _norm_answer(s["h"], s["o"], s["rstd_post"], s["rstd_pre"], s["q"], s["scales"])
        pt.pt_block_norm_bwd(s["dy"], s["dres"], s["x"], s["s"], s["post"], s["gate"], s["pre"], s["rstd_post"],
                             s["rstd_pre"], s["dx"], s["dresidual"], s["dgate"], s["dpost"], s["dpre"], R, C,
                             s["branch_scale"], s["residual_scale"], gate, stream[c["stream"]], 0,
                             workspace=s["workspace"])
        got = {"dx": s["dx"], "dresidual": s["dresidual"], "dpost": s["dpost"], "dpre": s["dpre"]}
        return dict(got, dgate=s["dgate"]) if c["gate"] != "none" else got
    T, H, k = c["rows"], c["cols"], c["k"]
    if op == "combine":
        pt.pt_moe_combine(s["y"], s["weights"], s["row_of"], s["base"], s["o"], T, T * k, H, k)
        return {"out": s["o"]}
    pt.pt_moe_combine_bwd(s["dout"], s["y"], s["weights"], s["row_of"], s["drows"], s["dweights"], T, T * k, H, k)
    return {"drows": s["drows"], "dweights": s["dweights"]}


def _norm_answer(h, y, rstd_post, rstd_pre, q, scales):
    """Codes and scale bytes as the eight-bit numbers they are."""
    got = {"residual_out": h, "y": y, "rstd_post": rstd_post, "rstd_pre": rstd_pre}
    if q is not None:
        got["q"] = q.view(torch.float8_e4m3fn)
        got["scales"] = scales.view(torch.float8_e8m0fnu) if scales.dtype == torch.uint8 else scales
    return got


def _act(c, act):
    if act == "none":
        return c
    if act == "relu2":
        return c.clamp(min=0).square()
    if act == "silu":
        return c / (1 + torch.exp(-c))
    if act == "gelu":
        return 0.5 * c * (1 + torch.erf(c * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * c * (1 + torch.tanh((2 / math.pi) ** 0.5 * (c + 0.044715 * c * c * c)))
    gate, up = c.chunk(2, 1)
    return gate / (1 + torch.exp(-gate)) * up


def _act_gradient(dh, c, act):
    if act == "none":
        return dh
    if act == "relu2":
        return dh * 2 * c.clamp(min=0)
    if act == "silu":
        p = 1 / (1 + torch.exp(-c))
        return dh * p * (1 + c * (1 - p))
    if act == "gelu":
        return dh * (0.5 * (1 + torch.erf(c * 0.5 ** 0.5)) + c * torch.exp(-0.5 * c * c) * (2 * math.pi) ** -0.5)
    if act == "gelu_tanh":
        b = (2 / math.pi) ** 0.5
        t = torch.tanh(b * (c + 0.044715 * c * c * c))
        return dh * (0.5 * (1 + t) + 0.5 * c * (1 - t * t) * b * (1 + 3 * 0.044715 * c * c))
    gate, up = c.chunk(2, 1)
    p = 1 / (1 + torch.exp(-gate))
    return torch.cat((dh * up * p * (1 + gate * (1 - p)), dh * gate * p), 1)


def _block_codes(v):
    """MXFP8 of v [R, C] (fp32): codes and scale bytes."""
    b = v.unflatten(1, (-1, 32))
    e = (torch.frexp(b.abs().amax(2))[1] - 9).clamp(min=-127)
    e = torch.where(b.abs().amax(2) > 0, e, -127)
    q = torch.ldexp(b, -e.unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn).flatten(1)
    return q.view(torch.uint8), (e + 127).to(torch.uint8)


def _row_codes(v):
    """E4M3 of v [R, C] (fp32) with one factor per row."""
    a = v.abs().amax(1)
    f = torch.where(a > 0, (448 / a).clamp(max=torch.finfo(F32).max), 1.0)
    q = (v * f.unsqueeze(1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), 1 / f


def _gate_of(s):
    """The gate as a factor of [R, C], in fp32."""
    kind = s["case"]["gate"]
    if kind == "none":
        return torch.ones((), device=s["x"].device)
    return s["gate"].unsqueeze(1) if kind == "rows" else s["gate"].float()


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "linear":
        v = s["x"].float() @ s["w"].float().t()
        if c["bias"]:
            v = v + s["bias"].float()
        out = _act(v, c["act"])
        if c["residual"]:
            out = s["residual"].float() + out
        out = out.to(_type(c))
        return {"out": out, "c": v.to(BF16)} if c["save"] else {"out": out}
    if op == "linear_dgrad":
        dh = s["dy"].float() @ s["w"].float()
        if c["act"] != "none":
            dh = _act_gradient(dh, s["c"].float(), c["act"])
        return {"dx": (dh + s["add"].float() if c["add"] else dh).to(BF16)}
    if op == "linear_wgrad":
        dy = s["dy"].float()
        got = {"dw": dy.t() @ s["x"].float()}
        return dict(got, dbias=dy.sum(0)) if c["bias"] else got
    if op == "block_norm":
        x, gate = s["x"].float(), _gate_of(s)
        rpost = torch.rsqrt(x.square().mean(1) + EPS)
        u = x * rpost.unsqueeze(1) * s["post"].float()
        h = (s["residual_scale"] * s["residual"].float() + s["branch_scale"] * gate * u).to(s["residual"].dtype)
        v = h.float()
        rpre = torch.rsqrt(v.square().mean(1) + EPS)
        v = v * rpre.unsqueeze(1) * s["pre"].float()
        q, scales = {"none": lambda t: (None, None), "mxfp8": _block_codes, "fp8rows": _row_codes}[c["codes"]](v)
        return _norm_answer(h, v.to(BF16), rpost, rpre, q, scales)
    if op == "block_norm_bwd":
        gate, kind = _gate_of(s), c["gate"]
        rpre, rpost = s["rstd_pre"].unsqueeze(1), s["rstd_post"].unsqueeze(1)
        hhat, dy = s["s"].float() * rpre, s["dy"].float()
        g = dy * s["pre"].float()
        ds = s["dres"].float() + rpre * (g - hhat * (g * hhat).mean(1, keepdim=True))
        xhat = s["x"].float() * rpost
        db = s["branch_scale"] * ds
        du = db * gate
        g = du * s["post"].float()
        dx = rpost * (g - xhat * (g * xhat).mean(1, keepdim=True))
        got = {"dx": dx.to(BF16), "dresidual": (s["residual_scale"] * ds).to(s["s"].dtype), "dpost": (du * xhat).sum(0),
               "dpre": (dy * hhat).sum(0)}
        if kind != "none":
            dgate = db * xhat * s["post"].float()
            got["dgate"] = {"cols": lambda: dgate.sum(0), "rows": lambda: dgate.sum(1), "full": lambda: dgate.to(BF16)}[kind]()
        return got
    T, k = c["rows"], c["k"]
    ok, row = s["row_of"] >= 0, s["row_of"].long().clamp(min=0)
    if op == "combine":
        out = s["base"].float() if c["base"] else torch.zeros((T, c["cols"]), device=s["y"].device)
        for j in range(k):
            y = torch.where(ok[:, j, None], s["y"].index_select(0, row[:, j]).float(), 0.0)
            out = out + (y * s["weights"][:, j, None] if c["weights"] else y)
        return {"out": out.to(BF16)}
    dout = s["dout"].float()
    drows = torch.zeros_like(s["y"])
    dweights = torch.empty((T, k), device=dout.device)
    for j in range(k):
        has = ok[:, j].nonzero().flatten()
        drows[row[has, j]] = (s["weights"][has, j, None] * dout[has]).to(BF16)
        dweights[:, j] = torch.where(ok[:, j], (s["y"].index_select(0, row[:, j]).float() * dout).sum(1), 0.0)
    return {"drows": drows, "dweights": dweights}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    R = case["rows"]
    if op.startswith("linear"):
        N, K = case["out"], case["in"]
        flops = 2 * R * N * K
        if op == "linear":
            o, size = N // _glu(case), 4 if case["stream"] == "f32" else 2
            more = 2 * N * case["bias"] + R * o * size * (1 + case["residual"]) + 2 * R * N * case["save"]
            return {"bytes": 2 * (R * K + N * K) + more, "flops": flops}
        if op == "linear_dgrad":
            extra = 2 * _glu(case) if case["act"] != "none" else 1 + case["add"]
            return {"bytes": 2 * (R * N + N * K + R * K * extra), "flops": flops}
        return {"bytes": 2 * R * (N + K) + 4 * N * K + 4 * N * case["bias"], "flops": flops}
    C = case["cols"]
    n = R * C
    if op.startswith("block_norm"):
        r, gate = 4 if case["stream"] == "f32" else 2, 2 if case["gate"] == "full" else 0
        if op == "block_norm":
            code = {"none": 0, "mxfp8": 1 + 1 / 32, "fp8rows": 1}[case["codes"]]
            return {"bytes": int(n * (2 + 2 * r + gate + 2 + code)) + 4 * C + 8 * R, "flops": 10 * n}
        return {"bytes": n * (2 + 3 * r + 2 + 2 + 2 * gate) + 12 * C + 8 * R, "flops": 24 * n}
    k = case["k"]
    if op == "combine":
        return {"bytes": 2 * n * (k + 1 + case["base"]) + R * k * (4 + 4 * case["weights"]), "flops": 2 * n * k}
    return {"bytes": 2 * n * (2 * k + 1) + 12 * R * k, "flops": 3 * n * k}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def d(name):
        return s[name].to(F64)

    if op == "linear":
        c = torch.mm(d("x"), d("w").t())
        if s["bias"] is not None:
            c += d("bias")
        out = _act_64(c, case["act"])
        if s["residual"] is not None:
            out = out + d("residual")
        return {"out": out, "c": c} if case["save"] else {"out": out}
    if op == "linear_dgrad":
        dx = torch.mm(d("dy"), d("w"))
        if case["act"] != "none":
            c = d("c").requires_grad_(True)
            dx = torch.autograd.grad(_act_64(c, case["act"]), c, dx)[0]
        return {"dx": dx + d("add") if s["add"] is not None else dx}
    if op == "linear_wgrad":
        got = {"dw": torch.mm(d("dy").t(), d("x"))}
        if case["bias"]:
            got["dbias"] = torch.mv(d("dy").t(), torch.ones(case["rows"], dtype=F64, device=s["dy"].device))
        return got
    if op == "block_norm":
        x = d("x")
        rpost = (x.pow(2).sum(1) / case["cols"] + EPS).pow(-0.5)
        branch = x * rpost[:, None] * d("post") * _gate_64(s, case)
        h = (d("residual") * s["residual_scale"] + branch * s["branch_scale"]).to(s["residual"].dtype).to(F64)
        rpre = (h.pow(2).sum(1) / case["cols"] + EPS).pow(-0.5)
        y = h * rpre[:, None] * d("pre")
        got = {"residual_out": h, "y": y, "rstd_post": rpost, "rstd_pre": rpre}
        if case["codes"] == "mxfp8":
            blocks = y.view(case["rows"], -1, 32)
            e = (torch.floor(torch.log2(blocks.abs().amax(2))) - 8).clamp(-127, 127)
            unit = torch.pow(torch.full_like(e, 2.0), e)
            got["q"], got["scales"] = _e4m3_64((blocks / unit[..., None]).reshape(y.shape)), unit
        elif case["codes"] == "fp8rows":
            factor = y.abs().amax(1) / 448
            got["q"], got["scales"] = _e4m3_64(y / factor[:, None]), factor
        return got
    if op == "block_norm_bwd":
        n, gate = case["cols"], _gate_64(s, case)
        rpre, rpost = d("rstd_pre")[:, None], d("rstd_post")[:, None]
        dy, stream, x, alpha = d("dy"), d("s"), d("x"), s["branch_scale"]
        gw = dy * d("pre") * rpre
        ds = d("dres") + gw - stream * rpre.pow(2) * ((gw * stream).sum(1, keepdim=True) / n)
        gx = ds * alpha * gate * d("post") * rpost
        dx = gx - x * rpost.pow(2) * ((gx * x).sum(1, keepdim=True) / n)
        got = {"dx": dx, "dresidual": s["residual_scale"] * ds,
               "dpost": (alpha * ds * gate * x * rpost).sum(0), "dpre": (dy * stream * rpre).sum(0)}
        if case["gate"] != "none":
            full = alpha * ds * x * rpost * d("post")
            got["dgate"] = full if case["gate"] == "full" else full.sum(0 if case["gate"] == "cols" else 1)
        return got
    T, H, k = case["rows"], case["cols"], case["k"]
    y = torch.cat((s["y"], torch.zeros((1, H), dtype=BF16, device=s["y"].device)))
    row = torch.where(s["row_of"] < 0, T * k, s["row_of"]).long()
    if op == "combine":
        out = d("base") if s["base"] is not None else torch.zeros((T, H), dtype=F64, device=y.device)
        for j in range(k):
            part = y[row[:, j]].to(F64)
            out += part * s["weights"][:, j:j + 1].to(F64) if s["weights"] is not None else part
        return {"out": out}
    drows = torch.zeros((T * k + 1, H), dtype=F64, device=y.device)
    dweights = torch.zeros((T, k), dtype=F64, device=y.device)
    for j in range(k):
        drows[row[:, j]] = d("dout") * s["weights"][:, j:j + 1].to(F64)
        dweights[:, j] = (d("dout") * y[row[:, j]].to(F64)).sum(1)
    return {"drows": drows[:-1], "dweights": dweights}


def _act_64(c, act):
    if act == "swiglu":
        half = c.shape[1] // 2
        return c[:, :half] * torch.sigmoid(c[:, :half]) * c[:, half:]
    return {"none": lambda: c, "relu2": lambda: torch.where(c > 0, c * c, torch.zeros_like(c)),
            "silu": lambda: c * torch.sigmoid(c), "gelu": lambda: c * 0.5 * torch.erfc(-c / math.sqrt(2)),
            "gelu_tanh": lambda: c * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (c + 0.044715 * c.pow(3)))}[act]()


def _gate_64(s, case):
    if case["gate"] == "none":
        return 1.0
    return s["gate"].to(F64)[:, None] if case["gate"] == "rows" else s["gate"].to(F64)


def _e4m3_64(v):
    """The nearest E4M3 number (ties to even, at most 448) to each of v, in 64 bits."""
    a = v.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.pow(torch.full_like(e, 2.0), e - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=448.0)
