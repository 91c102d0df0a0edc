"""Cases for the operators around the expert grouped GEMM: the residual RMS norm
with 8-bit outputs (forward and backward), the router (top-k, weights, expert
order; forward and backward) and the whole MoE layer for a few tokens.

Shapes follow the package's workloads: hidden size 4096 with 256 experts of
inner size 2048, six per token, and hidden and inner size 2880 with 32 experts,
four per token; 8192 and 16384 tokens for training, 1 to 64 for serving.
"""
import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # one decoded token: the latency of the norm before the router and FC1
        {"name": "norm_1_mxfp8", "op": "norm", "rows": 1, "cols": 4096, "stream": "bf16", "codes": "mxfp8"},
        # a training or prompt batch of 8192 tokens at hidden size 4096
        {"name": "norm_8192_mxfp8", "op": "norm", "rows": 8192, "cols": 4096, "stream": "bf16", "codes": "mxfp8"},
        # a ragged prompt at hidden size 2880, residual stream kept in fp32, one factor per row
        {"name": "norm_1021_fp8rows_f32", "op": "norm", "rows": 1021, "cols": 2880, "stream": "f32", "codes": "fp8rows"},
        # the training step's backward over 16384 tokens
        {"name": "norm_bwd_16384", "op": "norm_bwd", "rows": 16384, "cols": 2880, "stream": "bf16"},
        # a short ragged micro-batch with an fp32 gradient stream
        {"name": "norm_bwd_517_f32", "op": "norm_bwd", "rows": 517, "cols": 4096, "stream": "f32"},
        # decode: five tokens to 256 experts, sigmoid scores with a balancing bias
        {"name": "route_5_sigmoid", "op": "route", "tokens": 5, "experts": 256, "k": 6, "gate": "sigmoid", "renorm": True,
         "logits": "f32"},
        # training: 16384 tokens to 32 experts, softmax over the chosen four
        {"name": "route_16384_softmax", "op": "route", "tokens": 16384, "experts": 32, "k": 4, "gate": "softmax",
         "renorm": True, "logits": "bf16"},
        # the training step's backward over 8192 tokens and 256 experts
        {"name": "route_bwd_8192", "op": "route_bwd", "tokens": 8192, "experts": 256, "k": 6, "gate": "softmax",
         "renorm": False, "logits": "f32"},
        # one token through bf16 experts: the latency of decoding
        {"name": "few_1_bf16", "op": "few", "tokens": 1, "experts": 32, "hidden": 2880, "inner": 2880, "k": 4,
         "gate": "softmax", "renorm": True, "weights": "bf16"},
        # a small decode batch on 4-bit experts
        {"name": "few_7_mxfp4", "op": "few", "tokens": 7, "experts": 256, "hidden": 4096, "inner": 2048, "k": 6,
         "gate": "sigmoid", "renorm": True, "weights": "mxfp4"},
        # a decode batch that touches every one of 32 8-bit experts several times
        {"name": "few_33_mxfp8", "op": "few", "tokens": 33, "experts": 32, "hidden": 2880, "inner": 2880, "k": 4,
         "gate": "softmax", "renorm": True, "weights": "mxfp8"},
        # the largest batch: most of 256 bf16 experts are read
        {"name": "few_64_bf16", "op": "few", "tokens": 64, "experts": 256, "hidden": 4096, "inner": 2048, "k": 6,
         "gate": "sigmoid", "renorm": True, "weights": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """An odd multiple of 32: rows of it start at every place of a cache line."""
    return 32 * (_log_uniform(rng, lo, hi) | 1)


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "route", "route_bwd", "few", "few"])
    if op in ("norm", "norm_bwd"):
        c = {"op": op, "rows": _log_uniform(rng, 1, 16384), "cols": _width(rng, 8, 158),
             "stream": rng.choice(["bf16", "f32"])}
        if op == "norm":
            c["codes"] = rng.choice(["none", "mxfp8", "fp8rows"])
        return c
    experts = rng.choice([8, 32, 60, 128, 256])
    gate = rng.choice(["softmax", "sigmoid"])
    k = rng.randint(1, 8 if op != "few" else 6)
    renorm = k > 1 and rng.random() < 0.7  # of one chosen expert the share is 1, with no gradient
    if op in ("route", "route_bwd"):
        return {"op": op, "tokens": _log_uniform(rng, 1, 16384), "experts": experts, "k": min(k, experts - 2),
                "gate": gate, "renorm": renorm, "logits": rng.choice(["f32", "bf16"])}
    return {"op": op, "tokens": _log_uniform(rng, 1, 64), "experts": experts, "hidden": _width(rng, 16, 126),
            "inner": _width(rng, 16, 62), "k": k, "gate": gate, "renorm": renorm,
            "weights": rng.choice(["bf16", "mxfp8", "mxfp4"])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda" if torch.cuda.is_available() else "cpu")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=g.device) * std


def _stream_type(case):
    return torch.float32 if case["stream"] == "f32" else torch.bfloat16


def _logits(g, case, tokens):
    """Router logits: a token's part and an expert's, as a trained router gives them, with four experts shut (two of eight)."""
    E = case["experts"]
    z = _randn(g, tokens, E) + _randn(g, E, std=0.5)
    shut = torch.randperm(E, generator=g, device=g.device)[: 4 if E > 8 else 2]
    if E - len(shut) >= case["k"]:
        z[:, shut] = float("-inf")
    return z


def _quantised(w, kind):
    """Block-scaled codes and scale bytes of w [..., K]: 32 values to a power of two."""
    v = w.float().unflatten(-1, (-1, 32))
    top = 8 if kind == "mxfp8" else 2
    e = torch.frexp(v.abs().amax(-1))[1] - 1 - top
    v = torch.ldexp(v, -e.unsqueeze(-1)).flatten(-2)
    if kind == "mxfp8":
        codes = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
        n = torch.bucketize(v.abs(), edges).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        codes = n[..., 0::2] | (n[..., 1::2] << 4)
    return codes, (e + 127).to(torch.uint8)


def _experts(g, E, rows, cols, kind):
    """E weight matrices [rows, cols] of standard deviation cols^-1/2, made a few experts at a time."""
    step = max(1, (1 << 27) // (rows * cols))
    parts = [torch.randn((min(step, E - i), rows, cols), generator=g, device=g.device, dtype=torch.bfloat16).mul_(cols ** -0.5)
             for i in range(0, E, step)] if kind == "bf16" else None
    if parts is not None:
        out = torch.empty((E, rows, cols), dtype=torch.bfloat16, device=g.device)
        torch.cat(parts, out=out)
        return out, None
    width = cols if kind == "mxfp8" else cols // 2
    q = torch.empty((E, rows, width), dtype=torch.uint8, device=g.device)
    s = torch.empty((E, rows, cols // 32), dtype=torch.uint8, device=g.device)
    for i in range(0, E, step):
        n = min(step, E - i)
        q[i:i + n], s[i:i + n] = _quantised(_randn(g, n, rows, cols, std=cols ** -0.5), kind)
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    dev = g.device
    s = {"case": case, "op": case["op"]}
    bf16 = torch.bfloat16
    if case["op"] in ("norm", "norm_bwd"):
        R, C, dt = case["rows"], case["cols"], _stream_type(case)
        s["weight"] = (1 + _randn(g, C, std=0.2)).to(bf16)
        if case["op"] == "norm":
            s["x"] = _randn(g, R, C).to(bf16)
            s["residual"] = _randn(g, R, C, std=3.0).to(dt)
        else:
            s["s"] = _randn(g, R, C, std=3.0).to(dt)
            s["rstd"] = torch.rsqrt(s["s"].float().square().mean(1) + EPS)
            s["dy"] = _randn(g, R, C, std=1e-2).to(bf16)
            s["dres"] = _randn(g, R, C, std=1e-2).to(dt)
    else:
        T, E, k = case["tokens"], case["experts"], case["k"]
        z = _logits(g, case, T)
        s["logits"] = z.to(bf16) if case.get("logits") == "bf16" else z
        s["bias"] = _randn(g, E, std=0.05) if case["gate"] == "sigmoid" else None
        s["scale"] = 2.5 if case["gate"] == "sigmoid" else 1.0
        if case["op"] == "route_bwd":
            s["ids"] = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)[1][:, :k].to(torch.int32).contiguous()
            s["dweights"] = _randn(g, T, k)
        if case["op"] == "few":
            H, I = case["hidden"], case["inner"]
            s["x"] = _randn(g, T, H).to(bf16)
            s["w1"], s["w1_scale"] = _experts(g, E, 2 * I, H, case["weights"])
            s["w2"], s["w2_scale"] = _experts(g, E, H, I, case["weights"])
    if own:
        _buffers(s, case, dev)
    return s


def _buffers(s, case, dev):
    """The outputs and the workspace that a program on the package's caller-owned buffers keeps."""
    import moe_expert_grouped_gemm_amd as pt

    def new(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=dev)

    op = case["op"]
    if op == "norm":
        R, C = case["rows"], case["cols"]
        s["residual_out"], s["y"], s["rstd"] = new((R, C), _stream_type(case)), new((R, C), torch.bfloat16), new(R, torch.float32)
        s["q"] = new((R, C), torch.uint8) if case["codes"] != "none" else None
        s["scales"] = {"none": None, "mxfp8": new((R, C // 32), torch.uint8), "fp8rows": new(R, torch.float32)}[case["codes"]]
    elif op == "norm_bwd":
        R, C = case["rows"], case["cols"]
        s["ds"], s["dweight"] = new((R, C), _stream_type(case)), new(C, torch.float32)
        s["workspace"] = new(pt.pt_rmsnorm_workspace_size(R, C), torch.uint8)
    else:
        T, E, k = case["tokens"], case["experts"], case["k"]
        if op == "route_bwd":
            s["dlogits"] = torch.empty_like(s["logits"])
            return
        s["topk_ids"], s["topk_weights"] = new((T, k), torch.int32), new((T, k), torch.float32)
        if op == "route":
            s["lens"], s["row_of"], s["token_of"] = new(E, torch.int64), new((T, k), torch.int32), new(T * k, torch.int32)
            s["workspace"] = new(pt.pt_moe_route_workspace_size(T, E, k), torch.uint8)
        else:
            s["out"] = new((T, case["hidden"]), torch.bfloat16)
            s["workspace"] = new(pt.pt_moe_few_tokens_workspace_size(T, E, case["hidden"], case["inner"], k), torch.uint8)


# ------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import moe_expert_grouped_gemm_amd as pt
    c, op = s["case"], s["op"]
    stream = {"bf16": pt.PT_BF16, "f32": pt.PT_FP32}
    if op == "norm":
        codes = {"none": pt.PT_BF16, "mxfp8": pt.PT_MXFP8_E4M3, "fp8rows": pt.PT_FP8_E4M3_ROWWISE}[c["codes"]]
        pt.pt_rmsnorm_fwd(s["x"], s["residual"], s["weight"], s["residual_out"], s["y"], s["q"], s["scales"], s["rstd"],
                          c["rows"], c["cols"], EPS, stream[c["stream"]], codes)
        return _norm_answer(s["residual_out"], s["y"], s["rstd"], s["q"], s["scales"])
    if op == "norm_bwd":
        pt.pt_rmsnorm_bwd(s["dy"], s["s"], s["weight"], s["rstd"], s["dres"], s["ds"], s["dweight"], c["rows"], c["cols"],
                          stream[c["stream"]], 0, workspace=s["workspace"])
        return {"ds": s["ds"], "dweight": s["dweight"]}
    gate = pt.PT_GATE_SIGMOID if c["gate"] == "sigmoid" else pt.PT_GATE_SOFTMAX
    logits = stream[c.get("logits", "f32")]
    T, E, k, renorm = c["tokens"], c["experts"], c["k"], int(c["renorm"])
    if op == "route":
        pt.pt_moe_route(s["logits"], s["bias"], s["topk_ids"], s["topk_weights"], s["lens"], s["row_of"], s["token_of"],
                        T, E, k, logits, gate, renorm, s["scale"], workspace=s["workspace"])
        return {"ids": s["topk_ids"], "weights": s["topk_weights"], "lens": s["lens"], "row_of": s["row_of"],
                "token_of": s["token_of"]}
    if op == "route_bwd":
        pt.pt_moe_route_bwd(s["logits"], s["ids"], s["dweights"], s["dlogits"], T, E, k, logits, gate, renorm, s["scale"])
        return {"dlogits": s["dlogits"]}
    w = {"bf16": pt.PT_BF16, "mxfp8": pt.PT_MXFP8_E4M3, "mxfp4": pt.PT_MXFP4_E2M1}[c["weights"]]
    pt.pt_moe_few_tokens(s["x"], s["logits"], s["bias"], s["w1"], s["w1_scale"], s["w2"], s["w2_scale"], s["out"],
                         s["topk_ids"], s["topk_weights"], T, E, c["hidden"], c["inner"], k, logits, gate, renorm,
                         s["scale"], w, workspace=s["workspace"])
    return {"out": s["out"], "ids": s["topk_ids"], "weights": s["topk_weights"]}


def _norm_answer(residual_out, y, rstd, q, scales):
    """Codes and scale bytes as the eight-bit numbers they are."""
    got = {"residual_out": residual_out, "y": y, "rstd": rstd}
    if q is not None:
        got["q"] = q.view(torch.float8_e4m3fn)
        got["scales"] = scales.view(torch.float8_e8m0fnu) if scales.dtype == torch.uint8 else scales
    return got


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
    f = torch.where(a > 0, (448 / a).clamp(max=torch.finfo(torch.float32).max), 1.0)
    q = (v * f.unsqueeze(1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), 1 / f


def _choice(logits, bias, case, scale):
    """The chosen experts [T, k] and their weights, ties to the lower index; -inf is never chosen."""
    k = case["k"]
    z = logits.float()
    if case["gate"] == "sigmoid":
        value = torch.sigmoid(z.double())
        score = torch.where(z > float("-inf"), value + bias, float("-inf")).float()
    else:
        value, score = torch.softmax(z, 1), z
    top, ids = torch.sort(score, dim=1, descending=True, stable=True)
    ok = top[:, :k] > float("-inf")
    ids = ids[:, :k]
    w = torch.where(ok, value.gather(1, ids), 0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0)
    return torch.where(ok, ids, -1), (w * scale).float()


def _weights_of(w, scales, ids, kind):
    """The chosen experts' matrices [pairs, rows, cols] in fp32."""
    q = w.index_select(0, ids)
    if kind == "bf16":
        return q.float()
    if kind == "mxfp8":
        v = q.view(torch.float8_e4m3fn).float()
    else:
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=w.device)
        v = torch.stack((grid[(q & 15).int()], grid[(q >> 4).int()]), -1).flatten(-2)
    f = torch.ldexp(torch.ones((), device=w.device), scales.index_select(0, ids).int() - 127)
    return v.unflatten(-1, (-1, 32)).mul_(f.unsqueeze(-1)).flatten(-2)


def _run_plain(s):
    c, op = s["case"], s["op"]
    bf16 = torch.bfloat16
    if op == "norm":
        h = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
        v = h.float()
        rstd = torch.rsqrt(v.square().mean(1) + EPS)
        v = v * rstd.unsqueeze(1) * s["weight"].float()
        q, scales = {"none": lambda t: (None, None), "mxfp8": _block_codes, "fp8rows": _row_codes}[c["codes"]](v)
        return _norm_answer(h, v.to(bf16), rstd, q, scales)
    if op == "norm_bwd":
        v, dy, r = s["s"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
        g = dy * s["weight"].float()
        ds = s["dres"].float() + r * (g - v * (r * r * (g * v).mean(1, keepdim=True)))
        return {"ds": ds.to(s["s"].dtype), "dweight": (dy * v * r).sum(0)}
    if op == "route_bwd":
        return {"dlogits": _route_gradient(s, c).to(s["logits"].dtype)}
    ids, w = _choice(s["logits"], s["bias"], c, s["scale"])
    T, E, k = c["tokens"], c["experts"], c["k"]
    if op == "route":
        flat = torch.where(ids < 0, E, ids).flatten()
        order = torch.argsort(flat, stable=True)
        row_of = torch.empty_like(order)
        row_of[order] = torch.arange(T * k, device=order.device)
        lens = (flat.unsqueeze(1) == torch.arange(E, device=flat.device)).sum(0)
        used = torch.arange(T * k, device=flat.device) < lens.sum()
        return {"ids": ids.int(), "weights": w, "lens": lens, "row_of": torch.where(ids < 0, -1, row_of.view(T, k)).int(),
                "token_of": torch.where(used, order // k, -1).int()}
    pair = ids.flatten().clamp(min=0)
    x = s["x"].float().repeat_interleave(k, 0).unsqueeze(2)
    h = torch.bmm(_weights_of(s["w1"], s["w1_scale"], pair, c["weights"]), x).squeeze(2)
    gate, up = h.chunk(2, 1)
    h = gate / (1 + torch.exp(-gate)) * up
    y = torch.bmm(_weights_of(s["w2"], s["w2_scale"], pair, c["weights"]), h.unsqueeze(2)).view(T, k, -1)
    return {"out": (y * w.unsqueeze(2)).sum(1).to(bf16), "ids": ids.int(), "weights": w}


def _route_gradient(s, c):
    z, ids, g = s["logits"].float(), s["ids"].long(), s["dweights"] * s["scale"]
    if c["gate"] == "softmax":
        p = torch.softmax(z, 1)
        if not c["renorm"]:
            full = torch.zeros_like(z).scatter_(1, ids, g)
            return p * (full - (p * full).sum(1, keepdim=True))
        w = torch.softmax(z.gather(1, ids), 1)
        d = w * (g - (g * w).sum(1, keepdim=True))
    else:
        v = torch.sigmoid(z.gather(1, ids))
        if c["renorm"]:
            total = v.sum(1, keepdim=True)
            g = (g - (g * v).sum(1, keepdim=True) / total) / total
        d = g * v * (1 - v)
    return torch.zeros_like(z).scatter_(1, ids, d)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, r = case["rows"] * case["cols"], 4 if case["stream"] == "f32" else 2
        if op == "norm":
            code = {"none": 0, "mxfp8": 1 + 1 / 32, "fp8rows": 1}[case["codes"]]
            return {"bytes": int(n * (2 + r + r + 2 + code)) + 2 * case["cols"] + 4 * case["rows"], "flops": 5 * n}
        return {"bytes": n * (2 + r + r + r) + 6 * case["cols"] + 4 * case["rows"], "flops": 10 * n}
    T, E, k = case["tokens"], case["experts"], case["k"]
    size = 2 if case.get("logits") == "bf16" else 4
    if op == "route":
        return {"bytes": T * E * size + T * k * 16 + 8 * E, "flops": 8 * T * E}
    if op == "route_bwd":
        return {"bytes": 2 * T * E * size + T * k * 8, "flops": 8 * T * E}
    H, I = case["hidden"], case["inner"]
    per = {"bf16": 2, "mxfp8": 1 + 1 / 32, "mxfp4": 0.5 + 1 / 32}[case["weights"]]
    open_experts = E - (0 if E - (4 if E > 8 else 2) < k else 4 if E > 8 else 2)
    # experts that T tokens choosing k each are expected to meet, were all equally likely
    active = open_experts * (1 - (1 - k / open_experts) ** T)
    return {"bytes": int(active * 3 * H * I * per) + 4 * T * H + 4 * T * E + 8 * T * k, "flops": 6 * T * k * H * I}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "norm":
        h = (s["x"].to(f64) + s["residual"].to(f64)).to(s["residual"].dtype).to(f64)
        rstd = (h.pow(2).sum(1) / case["cols"] + EPS).pow(-0.5)
        y = h * rstd[:, None] * s["weight"].to(f64)
        got = {"residual_out": h, "y": y, "rstd": rstd}
        if case["codes"] == "mxfp8":
            blocks = y.view(case["rows"], -1, 32)
            e = (torch.floor(torch.log2(blocks.abs().amax(2))) - 8).clamp(-127, 127)
            unit = torch.pow(torch.full_like(e, 2.0), e)
            got["q"] = _e4m3_64((blocks / unit[..., None]).reshape(y.shape))
            got["scales"] = unit
        elif case["codes"] == "fp8rows":
            factor = y.abs().amax(1) / 448
            got["q"] = _e4m3_64(y / factor[:, None])
            got["scales"] = factor
        return got
    if op == "norm_bwd":
        v, dy, w, rows = s["s"].to(f64), s["dy"].to(f64), s["weight"].to(f64), case["cols"]
        inv = s["rstd"].to(f64)[:, None]
        xhat = v * inv
        gw = dy * w
        return {"ds": s["dres"].to(f64) + inv * gw - inv * xhat * ((gw * xhat).sum(1, keepdim=True) / rows),
                "dweight": torch.einsum("rc,rc->c", dy, xhat)}
    z = s["logits"].to(f64)
    T, E, k = case["tokens"], case["experts"], case["k"]
    if op == "route_bwd":
        ids = s["ids"].long()
        z = z.detach().clone().requires_grad_(True)
        prob = torch.softmax(z, 1) if case["gate"] == "softmax" else torch.sigmoid(z)
        chosen = torch.gather(prob, 1, ids)
        if case["renorm"]:
            chosen = chosen / chosen.sum(1, keepdim=True)
        (chosen * s["scale"] * s["dweights"].to(f64)).sum().backward()
        return {"dlogits": z.grad}
    shut = torch.isinf(z)
    prob = torch.softmax(z, 1) if case["gate"] == "softmax" else 1 / (1 + torch.exp(-z))
    score = z if case["gate"] == "softmax" else prob + s["bias"].to(f64)
    picked = torch.argsort(score.masked_fill(shut, -math.inf), dim=1, descending=True, stable=True)[:, :k]
    chosen = prob.gather(1, picked)
    if case["renorm"]:
        chosen = chosen / chosen.sum(1, keepdim=True)
    chosen = chosen * s["scale"]
    if op == "route":
        return {"ids": None, "weights": chosen, "lens": None, "row_of": None, "token_of": None}
    H, I, kind = case["hidden"], case["inner"], case["weights"]
    x, out = s["x"].to(f64), torch.zeros((T, H), dtype=f64, device=z.device)
    for e in torch.unique(picked).tolist():
        token, slot = torch.nonzero(picked == e, as_tuple=True)
        both = x[token] @ _matrix_64(s["w1"], s["w1_scale"], e, kind).t()
        h = both[:, :I] * torch.sigmoid(both[:, :I]) * both[:, I:]
        out.index_add_(0, token, (h @ _matrix_64(s["w2"], s["w2_scale"], e, kind).t()) * chosen[token, slot][:, None])
    return {"out": out, "ids": None, "weights": chosen}


def _e4m3_64(v):
    """The nearest E4M3 number (ties to even, at most 448) to each of v, in 64 bits."""
    a = v.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.pow(torch.full_like(e, 2.0), e - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=448.0)


def _matrix_64(w, scales, e, kind):
    if kind == "bf16":
        return w[e].double()
    if kind == "mxfp8":
        code = w[e].to(torch.int32)
        m, x = (code & 7).double(), (code >> 3) & 15
        v = torch.where(x > 0, (8 + m) * torch.pow(2.0, (x - 10).double()), m * 2.0 ** -9)
        v = torch.where(code >= 128, -v, v)
    else:
        code = torch.stack((w[e] & 15, w[e] >> 4), -1).flatten(1).to(torch.int32)
        m, x = (code & 1).double(), (code >> 1) & 3
        v = torch.where(x > 0, (2 + m) * torch.pow(2.0, (x - 2).double()), m * 0.5)
        v = torch.where(code >= 8, -v, v)
    unit = torch.pow(2.0, scales[e].double() - 127)
    return v * unit.repeat_interleave(32, 1)
