"""The norms around a block with its gate and residual scale, on the GPU against
the formulas in 64 bits.

Tolerances, derived.  A sum of `cols` squares or products is a tree at most 40
deep: 40 * 2^-24 of the sum of the terms' sizes.  rstd takes half of that and
three roundings: 24 * 2^-24 < 2e-6.  h is a sum of two products of which the
branch holds rstd and four roundings: 2.4e-6 of the branch and 2^-23 of the
whole, then half a step of the stream's type.  v from the stream that came out is
rstd and two roundings, y and codes its one rounding more.  In the backward, ds
is dres + rstd (g - shat m): four roundings of each term, and m within 40 * 2^-24
of mean |g shat|; e follows from ds with four roundings, dx is its like.  Sums
over rows: 2^-24 times the rows of a part, the 16-deep join of parts and the
terms' own error, of the sum of the terms' sizes.
"""
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm

pytestmark = pytest.mark.gpu

F64, BF16, F32 = torch.float64, torch.bfloat16, torch.float32
EPS = 1e-5
U = 2.0 ** -24
CODES = {"none": ptm.PT_BF16, "mxfp8": ptm.PT_MXFP8_E4M3, "rows": ptm.PT_FP8_E4M3_ROWWISE}
STREAM = {"bf16": (ptm.PT_BF16, BF16, 2.0 ** -8), "f32": (ptm.PT_FP32, F32, U)}
GATES = {"none": ptm.PT_BLOCK_GATE_NONE, "cols": ptm.PT_BLOCK_GATE_COLS, "rows": ptm.PT_BLOCK_GATE_ROWS,
         "full": ptm.PT_BLOCK_GATE_FULL}


def make(dev, rows, cols, stream, gate, seed, post=True, pre=True):
    g = torch.Generator(device=dev).manual_seed(seed)

    def n(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev) * std

    t = STREAM[stream][1]
    s = {"x": n(rows, cols, std=2.0).to(BF16), "residual": n(rows, cols, std=3.0).to(t), "stream": stream, "kind": gate,
         "post": (1 + n(cols, std=0.2)).to(BF16) if post else None, "pre": (1 + n(cols, std=0.2)).to(BF16) if pre else None,
         "gate": {"none": None, "cols": (0.5 + n(cols, std=0.2)).to(BF16), "rows": n(rows), "full": n(rows, cols).to(BF16)}[gate],
         "alpha": 0.7, "beta": 1.3}
    s["dy"], s["dres"] = n(rows, cols).to(BF16) if pre else None, n(rows, cols).to(t)
    return s


def gate64(s):
    if s["kind"] == "none":
        return torch.ones((), dtype=F64, device=s["x"].device)
    return s["gate"].to(F64)[:, None] if s["kind"] == "rows" else s["gate"].to(F64)


def forward(s, codes="none", with_y=True, residual_out=None):
    rows, cols = s["x"].shape
    dev, st = s["x"].device, STREAM[s["stream"]]
    pre = s["pre"] is not None
    o = {"h": residual_out if residual_out is not None else torch.full((rows, cols), 7.0, dtype=st[1], device=dev),
         "y": torch.full((rows, cols), 7.0, dtype=BF16, device=dev) if with_y and pre else None,
         "rpost": torch.full((rows,), 7.0, device=dev) if s["post"] is not None else None,
         "rpre": torch.full((rows,), 7.0, device=dev) if pre else None, "q": None, "scales": None}
    if codes != "none":
        o["q"] = torch.full((rows, cols), 0xEE, dtype=torch.uint8, device=dev)
        o["scales"] = (torch.full((rows, cols // 32), 0xEE, dtype=torch.uint8, device=dev) if codes == "mxfp8"
                       else torch.full((rows,), 7.0, device=dev))
    ptm.pt_block_norm_fwd(s["x"], s["residual"], s["post"], s["gate"], s["pre"], o["h"], o["y"], o["q"], o["scales"],
                          o["rpost"], o["rpre"], rows, cols, EPS, s["alpha"], s["beta"], GATES[s["kind"]], st[0], CODES[codes])
    torch.cuda.synchronize()
    return o


def check_forward(s, codes, o):
    half = STREAM[s["stream"]][2]
    x = s["x"].to(F64)
    rpost = (x.square().mean(1) + EPS).pow(-0.5)
    if s["post"] is not None:
        assert ((o["rpost"].to(F64) - rpost).abs() <= 2e-6 * rpost).all()
        x = x * rpost[:, None] * s["post"].to(F64)
    # the scales reach the kernel as fp32
    alpha, beta = torch.tensor([s["alpha"], s["beta"]], dtype=F32).to(F64).tolist()
    branch, stay = alpha * gate64(s) * x, beta * s["residual"].to(F64)
    h = branch + stay
    off = 2.4e-6 * branch.abs() + 2.0 ** -23 * (stay.abs() + h.abs())
    assert ((o["h"].to(F64) - h).abs() <= half * (h.abs() + off) + off).all()
    if s["pre"] is None:
        return
    h = o["h"].to(F64)
    rpre = (h.square().mean(1) + EPS).pow(-0.5)
    assert ((o["rpre"].to(F64) - rpre).abs() <= 2e-6 * rpre).all()
    v = h * rpre[:, None] * s["pre"].to(F64)
    if o["y"] is not None:
        assert ((o["y"].to(F64) - v).abs() <= (2.0 ** -8 + 3e-6) * v.abs() + 2.0 ** -134).all()
    if codes == "none":
        return
    deq = o["q"].view(torch.float8_e4m3fn).to(F64)
    if codes == "mxfp8":
        amax = v.unflatten(1, (-1, 32)).abs().amax(2)
        e = torch.floor(torch.log2(amax)) - 8
        have = o["scales"].to(F64) - 127
        edge = ((torch.log2(amax) - torch.round(torch.log2(amax))).abs() < 6e-6) & ((have - e).abs() == 1)
        assert ((have == e) | edge).all()
        unit = torch.pow(torch.full_like(have, 2.0), have).repeat_interleave(32, 1)
    else:
        factor = v.abs().amax(1) / 448
        assert ((o["scales"].to(F64) - factor).abs() <= 4e-6 * factor).all()
        unit = o["scales"].to(F64)[:, None]
    want = (v / unit).clamp(-448, 448)
    assert ((deq - want).abs() <= (2.0 ** -4 + 1e-5) * want.abs() + 2.0 ** -10).all()


SHAPES = [(1, 8), (1, 4096), (3, 40), (5, 2880), (64, 2880), (7, 5056), (33, 288), (9, 544), (2, 2048), (2, 2056), (3, 6144),
          (2, 8192), (2, 8224), (3, 16384), (1030, 544)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("stream", list(STREAM))
@pytest.mark.parametrize("gate", list(GATES))
def test_forward(dev, rows, cols, stream, gate):
    s = make(dev, rows, cols, stream, gate, rows * 7 + cols)
    check_forward(s, "none", forward(s))


@pytest.mark.parametrize("rows,cols", [(1, 4096), (5, 288), (3, 2880), (2, 8224), (700, 544)])
@pytest.mark.parametrize("stream", list(STREAM))
@pytest.mark.parametrize("codes", ["mxfp8", "rows"])
def test_codes(dev, rows, cols, stream, codes):
    s = make(dev, rows, cols, stream, "cols", rows + cols)
    o = forward(s, codes)
    check_forward(s, codes, o)
    bare = forward(s, codes, with_y=False)
    assert torch.equal(bare["q"], o["q"]) and torch.equal(bare["scales"], o["scales"])


@pytest.mark.parametrize("post,pre", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("stream", list(STREAM))
def test_one_norm_or_none(dev, post, pre, stream):
    for gate in GATES:
        s = make(dev, 6, 320, stream, gate, 5, post, pre)
        check_forward(s, "none", forward(s))
        check_backward(s, backward(s), 0)


def test_stream_in_place_and_the_plain_norm(dev):
    s = make(dev, 6, 320, "f32", "full", 5)
    own = s["residual"].clone()
    whole = forward(s)
    o = forward(dict(s, residual=own), residual_out=own)
    assert torch.equal(own, whole["h"]) and torch.equal(o["y"], whole["y"])
    # without gate, scales and norm after the block it is the residual norm, bit for bit
    for stream in STREAM:
        s = make(dev, 9, 2880, stream, "none", 6, post=False)
        s["alpha"] = s["beta"] = 1.0
        o = forward(s, "rows")
        h, y = torch.empty_like(o["h"]), torch.empty_like(o["y"])
        q, scales, rstd = torch.empty_like(o["q"]), torch.empty_like(o["scales"]), torch.empty_like(o["rpre"])
        ptm.pt_rmsnorm_fwd(s["x"], s["residual"], s["pre"], h, y, q, scales, rstd, 9, 2880, EPS, STREAM[stream][0],
                           ptm.PT_FP8_E4M3_ROWWISE)
        for a, b in ((h, o["h"]), (y, o["y"]), (q, o["q"]), (scales, o["scales"]), (rstd, o["rpre"])):
            assert torch.equal(a, b)


@pytest.mark.parametrize("codes", list(CODES))
def test_zero_nan_and_infinite_rows(dev, codes):
    s = make(dev, 6, 256, "f32", "rows", 9)
    s["x"][0], s["residual"][0] = 0, 0
    s["x"][1], s["residual"][1] = s["x"][1] * 0, s["residual"][1] * 1e-20
    s["x"][2, 7] = float("nan")
    s["residual"][3, 9] = float("inf")
    s["gate"][4] = float("nan")
    clean = make(dev, 6, 256, "f32", "rows", 9)
    o, ref = forward(s, codes), forward(clean, codes)
    assert torch.isfinite(o["y"][:2]).all() and (o["y"][0] == 0).all() and (o["h"][0] == 0).all()
    for r in (2, 3, 4):
        assert torch.isnan(o["y"][r].float()).any()
    for k in ("h", "y", "q", "scales"):
        if o[k] is not None:
            assert torch.equal(o[k][5], ref[k][5])


# ------------------------------------------------------------------ backward
def backward(s, accumulate=0, start=None, wanted=("dgate", "dpost", "dpre"), dresidual=None):
    rows, cols = s["x"].shape
    dev, st = s["x"].device, STREAM[s["stream"]]
    rpost = (s["x"].to(F64).square().mean(1) + EPS).pow(-0.5).to(F32)
    rpre = (s["residual"].to(F64).square().mean(1) + EPS).pow(-0.5).to(F32)
    start = start or {}
    o = {"dx": torch.full((rows, cols), 7.0, dtype=BF16, device=dev),
         "dresidual": torch.full((rows, cols), 7.0, dtype=st[1], device=dev) if dresidual is None else dresidual}
    shape = {"cols": ((cols,), F32), "rows": ((rows,), F32), "full": ((rows, cols), BF16)}.get(s["kind"])
    o["dgate"] = start.get("dgate", torch.full(shape[0], 7.0, dtype=shape[1], device=dev)) if shape and "dgate" in wanted else None
    for name, w in (("dpost", "post"), ("dpre", "pre")):
        o[name] = start.get(name, torch.full((cols,), 7.0, device=dev)) if s[w] is not None and name in wanted else None
    ws = torch.full((ptm.pt_block_norm_workspace_size(rows, cols),), 0xFF, dtype=torch.uint8, device=dev)
    pre, post = s["pre"] is not None, s["post"] is not None
    # the residual of the case stands for the forward's stream
    ptm.pt_block_norm_bwd(s["dy"], s["dres"], s["x"], s["residual"] if pre else None, s["post"], s["gate"], s["pre"],
                          rpost if post else None, rpre if pre else None, o["dx"], o["dresidual"], o["dgate"], o["dpost"],
                          o["dpre"], rows, cols, s["alpha"], s["beta"], GATES[s["kind"]], st[0], accumulate, workspace=ws)
    torch.cuda.synchronize()
    return dict(o, rpost=rpost, rpre=rpre)


def check_backward(s, o, start):
    half = STREAM[s["stream"]][2]
    rows, cols = s["x"].shape
    alpha, beta = torch.tensor([s["alpha"], s["beta"]], dtype=F32).to(F64).tolist()
    d = s["dres"].to(F64) if s["dres"] is not None else torch.zeros((rows, cols), dtype=F64, device=s["x"].device)
    size = d.abs()
    off = torch.zeros_like(d)
    if s["pre"] is not None:
        r = o["rpre"].to(F64)[:, None]
        shat, dy = s["residual"].to(F64) * r, s["dy"].to(F64)
        g = dy * s["pre"].to(F64)
        m, mabs = (g * shat).mean(1, keepdim=True), (g * shat).abs().mean(1, keepdim=True)
        d = d + r * (g - shat * m)
        off = 8 * U * (size + r * (g.abs() + (shat * m).abs())) + 48 * U * r * shat.abs() * mabs
        if o["dpre"] is not None:
            want, terms = start + (dy * shat).sum(0), start + (dy * shat).abs().sum(0)
            assert ((o["dpre"].to(F64) - want).abs() <= (rows / 64 + 40) * U * terms).all()
    want = beta * d
    o2 = beta * off + 2 * U * want.abs()
    assert ((o["dresidual"].to(F64) - want).abs() <= half * (want.abs() + o2) + o2).all()
    rp = o["rpost"].to(F64)[:, None] if s["post"] is not None else torch.ones((), dtype=F64, device=d.device)
    wp = s["post"].to(F64) if s["post"] is not None else torch.ones((), dtype=F64, device=d.device)
    gate = gate64(s)
    xhat = s["x"].to(F64) * rp
    t, toff = alpha * d * xhat, alpha * (off + 4 * U * d.abs()) * xhat.abs()
    e = alpha * d * gate * wp
    eoff = (gate * wp).abs() * alpha * (off + 6 * U * d.abs())
    dx, doff = e, eoff
    if s["post"] is not None:
        m, mabs = (e * xhat).mean(1, keepdim=True), (e * xhat).abs().mean(1, keepdim=True)
        dx = rp * (e - xhat * m)
        doff = rp * (eoff + xhat.abs() * (eoff * xhat.abs()).mean(1, keepdim=True) + 8 * U * (e.abs() + (xhat * m).abs()) +
                     48 * U * xhat.abs() * mabs)
    assert ((o["dx"].to(F64) - dx).abs() <= 2.0 ** -8 * (dx.abs() + doff) + doff + 1e-30).all()
    deep = (rows / 64 + 48) * U
    if o["dpost"] is not None:
        want, terms, more = start + (gate * t).sum(0), start + (gate * t).abs().sum(0), (gate.abs() * toff).sum(0)
        assert ((o["dpost"].to(F64) - want).abs() <= deep * terms + more).all()
    if o["dgate"] is None:
        return
    full, more = t * wp, toff * wp.abs()
    if s["kind"] == "full":
        assert ((o["dgate"].to(F64) - full).abs() <= 2.0 ** -8 * (full.abs() + more) + more + 4 * U * full.abs() + 1e-30).all()
    else:
        dim = 0 if s["kind"] == "cols" else 1
        base = start if s["kind"] == "cols" else 0
        want = base + full.sum(dim)
        bound = (deep if dim == 0 else 48 * U) * (base + full.abs().sum(dim)) + more.sum(dim)
        assert ((o["dgate"].to(F64) - want).abs() <= bound).all()


@pytest.mark.parametrize("rows,cols", SHAPES + [(300, 4064), (2100, 264)])
@pytest.mark.parametrize("stream", list(STREAM))
@pytest.mark.parametrize("gate", list(GATES))
def test_backward(dev, rows, cols, stream, gate):
    s = make(dev, rows, cols, stream, gate, rows * 5 + cols)
    check_backward(s, backward(s), 0)


@pytest.mark.parametrize("gate", list(GATES))
def test_accumulate_and_optional_gradients(dev, gate):
    s = make(dev, 70, 544, "bf16", gate, 12)
    first = backward(s)
    start = {k: torch.full((544,), 2.0, device=dev) for k in ("dpost", "dpre")}
    if gate == "cols":
        start["dgate"] = torch.full((544,), 2.0, device=dev)
    o = backward(s, 1, start)
    check_backward(s, o, 2.0)
    for drop in ("dgate", "dpost", "dpre"):
        o = backward(s, wanted=[n for n in ("dgate", "dpost", "dpre") if n != drop])
        for k in ("dx", "dresidual", "dgate", "dpost", "dpre"):
            assert o[k] is None or torch.equal(o[k], first[k]), k
    o = backward(s, wanted=())
    assert torch.equal(o["dx"], first["dx"]) and torch.equal(o["dresidual"], first["dresidual"])
    # no gradient past the next block, and the stream's gradient in place
    check_backward(dict(s, dres=None), backward(dict(s, dres=None)), 0)
    own = s["dres"].clone()
    o = backward(dict(s, dres=own), dresidual=own)
    assert torch.equal(own, first["dresidual"])


def test_no_rows(dev):
    s = make(dev, 0, 64, "bf16", "cols", 1)
    forward(s)
    o = backward(s)
    assert (o["dpost"] == 0).all() and (o["dpre"] == 0).all() and (o["dgate"] == 0).all()
    start = {k: torch.full((64,), 2.0, device=dev) for k in ("dpost", "dpre", "dgate")}
    o = backward(s, 1, start)
    assert (o["dpost"] == 2).all() and (o["dgate"] == 2).all()


def test_backward_by_differences(dev):
    """The gradients of the forward kernel itself: central differences of sum(y dy) + sum(h dres) along random
    directions, fp32 stream.  The forward is off by 2^-8 of y an element (its rounding), which over n elements adds like a
    random walk; the step is large enough that this is a few percent of the difference at most, and small enough that the
    third derivative is too."""
    s = make(dev, 64, 2880, "f32", "full", 21)
    s["residual"] = s["residual"] * 1.0
    stream = forward(s)["h"]

    def loss(inp):
        o = forward(inp)
        return (o["y"].to(F64) * s["dy"].to(F64)).sum() + (o["h"].to(F64) * s["dres"].to(F64)).sum()

    grads = backward(dict(s, residual=stream))
    g = torch.Generator(device=dev).manual_seed(2)
    for name, out in (("x", "dx"), ("residual", "dresidual"), ("gate", "dgate"), ("post", "dpost"), ("pre", "dpre")):
        # a step along the gradient, in values that the type holds
        d = grads[out].to(F64)
        step = 0.03 * s[name].to(F64).abs().mean() / d.abs().mean()
        up, down = (s[name].to(F64) + step * d).to(s[name].dtype), (s[name].to(F64) - step * d).to(s[name].dtype)
        got = loss(dict(s, **{name: up})) - loss(dict(s, **{name: down}))
        want = (d * (up.to(F64) - down.to(F64))).sum()
        noise = 4 * 2.0 ** -8 * (s["dy"].to(F64) ** 2).sum().sqrt()
        assert (got - want).abs() <= 0.02 * want.abs() + noise, name


def test_repeats_streams_and_graph(dev):
    s = make(dev, 1500, 1056, "bf16", "cols", 30)
    first, grad = forward(s, "mxfp8"), backward(s)
    for _ in range(3):
        again, gradn = forward(s, "mxfp8"), backward(s)
        for a, b in ((first, again), (grad, gradn)):
            assert all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)
    rows, cols = s["x"].shape
    ws = torch.empty(ptm.pt_block_norm_workspace_size(rows, cols), dtype=torch.uint8, device=dev)
    o = {k: torch.empty_like(v) for k, v in first.items()}
    b = {k: torch.empty_like(grad[k]) for k in ("dx", "dresidual", "dgate", "dpost", "dpre")}

    def run():
        ptm.pt_block_norm_fwd(s["x"], s["residual"], s["post"], s["gate"], s["pre"], o["h"], o["y"], o["q"], o["scales"],
                              o["rpost"], o["rpre"], rows, cols, EPS, s["alpha"], s["beta"], GATES["cols"], ptm.PT_BF16,
                              ptm.PT_MXFP8_E4M3)
        ptm.pt_block_norm_bwd(s["dy"], s["dres"], s["x"], s["residual"], s["post"], s["gate"], s["pre"], grad["rpost"],
                              grad["rpre"], b["dx"], b["dresidual"], b["dgate"], b["dpost"], b["dpre"], rows, cols, s["alpha"],
                              s["beta"], GATES["cols"], ptm.PT_BF16, 0, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        assert all(torch.equal(o[k], first[k]) for k in o) and all(torch.equal(b[k], grad[k]) for k in b)
        for t in [*o.values(), *b.values()]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
    assert all(torch.equal(o[k], first[k]) for k in o) and all(torch.equal(b[k], grad[k]) for k in b)
