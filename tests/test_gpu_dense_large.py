"""The dense operators where offsets pass 32 bits, and where calls run side by side.

The large matrices repeat P rows.  With small integers as operands the products
are exact in fp32 (sums below 2^24), and the elementwise rest of a row depends on
that row alone, so that outputs repeat too: bit for bit, and bit for bit those of
a call of the P rows, which the tests of ordinary sizes hold against 64 bits."""
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm
import test_gpu_block_norm as norms
import test_gpu_combine as joins
import test_gpu_linear as products
from test_gpu_linear import BF16, F32, F64, gen, ints, randn

pytestmark = pytest.mark.gpu

P, TIMES, COLS = 1000, 933, 2304                              # 933000 x 2304: more than 2^31 elements
assert P * TIMES * COLS > 1 << 31


def same(large, small):
    return torch.equal(large.view(TIMES, *small.shape), small.expand(TIMES, *small.shape))


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def test_forward(dev):
    g = gen(dev, 1)
    x, w, bias = ints(g, P, COLS, top=1), ints(g, COLS, COLS, top=1), ints(g, COLS)
    r = ints(g, P, COLS)
    for act, n in (("relu2", COLS), ("none", COLS)):
        small, saved = products.forward(x, w, bias, r, act=act, save=True)
        want = x.float() @ w.float().t() + bias.float()
        assert torch.equal(saved, want.to(BF16))
        out, c = products.forward(x.repeat(TIMES, 1), w, bias, r.repeat(TIMES, 1), act=act, save=True)
        assert same(out, small) and same(c, saved)
        del out, c


def test_forward_swiglu_and_fp32(dev):
    g = gen(dev, 2)
    x, w = ints(g, P, 40, top=1), ints(g, 2 * COLS, 40, top=1)
    small, saved = products.forward(x, w, out_type=F32, act="swiglu", save=True)
    out, c = products.forward(x.repeat(TIMES, 1), w, out_type=F32, act="swiglu", save=True)
    assert same(out, small) and same(c, saved)


def test_dgrad(dev):
    g = gen(dev, 3)
    dy, w, add = ints(g, P, COLS, top=1), ints(g, COLS, COLS, top=1), ints(g, P, COLS)
    small = products.dgrad(dy, w, add=add)
    assert torch.equal(small, (dy.float() @ w.float() + add.float()).to(BF16))
    big = add.repeat(TIMES, 1)
    assert same(products.dgrad(dy.repeat(TIMES, 1), w, add=big, dx=big), small)
    c = randn(g, P, 2 * COLS)
    small = products.dgrad(dy, w, c, act="swiglu")
    assert same(products.dgrad(dy.repeat(TIMES, 1), w, c.repeat(TIMES, 1), act="swiglu"), small)


def test_wgrad(dev):
    g = gen(dev, 4)
    x, dy = ints(g, P, COLS, top=1), ints(g, P, COLS, top=1)
    dw, db = products.wgrad(x.repeat(TIMES, 1), dy.repeat(TIMES, 1))
    assert torch.equal(dw, TIMES * (dy.float().t() @ x.float()))
    assert torch.equal(db, TIMES * dy.float().sum(0))


def test_act_bwd(dev):
    g = gen(dev, 5)
    c = randn(g, P, COLS)
    for act, cols in (("gelu_tanh", COLS), ("swiglu", COLS // 2)):
        dout = randn(g, P, cols)
        small = torch.empty_like(c)
        ptm.pt_linear_act_bwd(dout, c, small, P, COLS, products.ACTS[act])
        big = c.repeat(TIMES, 1)
        ptm.pt_linear_act_bwd(dout.repeat(TIMES, 1), big, big, P * TIMES, COLS, products.ACTS[act])
        assert same(big, small)


@pytest.mark.parametrize("stream,gate", [("bf16", "full"), ("f32", "rows")])
def test_block_norm(dev, stream, gate):
    one = norms.make(dev, P, COLS, stream, gate, 6)
    many = {k: v.repeat(TIMES, *[1] * (v.dim() - 1)) if torch.is_tensor(v) and len(v) == P else v for k, v in one.items()}
    for codes in ("none", "mxfp8", "rows"):
        small = norms.forward(one, codes)
        o = norms.forward(many, codes)
        assert all(same(o[k], small[k]) for k in o if o[k] is not None), codes
        del o
    small = norms.backward(one)
    rows, cols = many["x"].shape
    t = norms.STREAM[stream]
    dx, dr = torch.empty((rows, cols), dtype=BF16, device=dev), many["dres"]
    dg = torch.empty_like(many["gate"])
    dpost, dpre = torch.empty(cols, device=dev), torch.empty(cols, device=dev)
    ws = torch.empty(ptm.pt_block_norm_workspace_size(rows, cols), dtype=torch.uint8, device=dev)
    ptm.pt_block_norm_bwd(many["dy"], dr, many["x"], many["residual"], many["post"], many["gate"], many["pre"],
                          small["rpost"].repeat(TIMES), small["rpre"].repeat(TIMES), dx, dr, dg, dpost, dpre, rows, cols,
                          one["alpha"], one["beta"], norms.GATES[gate], t[0], 0, workspace=ws)
    assert same(dx, small["dx"]) and same(dr, small["dresidual"])
    # a gate per token: its sum over columns meets in the same order whatever the rows
    assert same(dg, small["dgate"])
    # sums over rows: additions of a part's rows and of the join, each 2^-24 of the terms' sizes
    shat = one["residual"].to(F64) * small["rpre"].to(F64)[:, None]
    terms = one["dy"].to(F64) * shat
    off = (rows / (ws.numel() // (8 * cols)) + 64) * 2.0 ** -24 * TIMES * terms.abs().sum(0)
    assert ((dpre.to(F64) - TIMES * terms.sum(0)).abs() <= off).all()


def test_joins(dev):
    """Rows, tokens and gradients past 2^31 elements: every row's own token, shifted by one."""
    g = gen(dev, 7)
    H = COLS
    T = P * TIMES
    rows, base = ints(g, P, H), ints(g, P, H)
    row_of = ((torch.arange(T, device=dev) + 1) % T).int().view(T, 1)
    w = torch.full((T, 1), 2.0, device=dev)
    big, out = rows.repeat(TIMES, 1), torch.empty((T, H), dtype=BF16, device=dev)
    ptm.pt_moe_combine(big, w, row_of, base.repeat(TIMES, 1), out, T, T, H, 1)
    assert same(out, 2 * rows.roll(-1, 0) + base)
    dw = torch.empty((T, 1), device=dev)
    ptm.pt_moe_combine_bwd(out, big, w, row_of, big, dw, T, T, H, 1)
    dout = 2 * rows.roll(-1, 0) + base
    assert same(big, (2 * dout).roll(1, 0))
    assert same(dw, (dout.float() * rows.roll(-1, 0).float()).sum(1, keepdim=True))


def case(dev, seed):
    """One run of the operators on outputs and workspaces of its own."""
    g = gen(dev, seed)
    M, N, K, k = 700 + 100 * seed, 264, 1032, 3
    x, w, dy = ints(g, M, K), ints(g, N, K), ints(g, M, N)
    s = norms.make(dev, M, K, "bf16", "cols", seed)
    j = joins.make(dev, M, K, k, seed)
    f = norms.backward(s)
    e = lambda *shape, dtype=F32: torch.full(shape, 7.0, dtype=dtype, device=dev)
    out = [e(M, N), e(M, K, dtype=BF16), e(N, K), e(N), e(M, K, dtype=BF16), e(M, K, dtype=BF16), e(K), e(K), e(K),
           e(M, K, dtype=BF16), e(j["M"], K, dtype=BF16), e(M, k)]
    ws = [products.workspace(op, M, N, K, dev) for op in (ptm.PT_OP_FWD, ptm.PT_OP_DGRAD, ptm.PT_OP_WGRAD)]
    ws.append(torch.empty(ptm.pt_block_norm_workspace_size(M, K), dtype=torch.uint8, device=dev))

    def run():
        ptm.pt_linear_fwd(x, w, None, None, out[0], None, M, N, K, out_dtype=ptm.PT_FP32, workspace=ws[0])
        ptm.pt_linear_dgrad(dy, w, None, None, out[1], M, N, K, workspace=ws[1])
        ptm.pt_linear_wgrad(x, dy, out[2], out[3], M, N, K, 0, workspace=ws[2])
        ptm.pt_block_norm_bwd(s["dy"], s["dres"], s["x"], s["residual"], s["post"], s["gate"], s["pre"], f["rpost"], f["rpre"],
                              out[4], out[5], out[6], out[7], out[8], M, K, s["alpha"], s["beta"], norms.GATES["cols"],
                              ptm.PT_BF16, 0, workspace=ws[3])
        ptm.pt_moe_combine(j["rows"], j["weights"], j["row_of"], j["base"], out[9], M, j["M"], K, k)
        ptm.pt_moe_combine_bwd(j["dout"], j["rows"], j["weights"], j["row_of"], out[10], out[11], M, j["M"], K, k)
    return run, out


def test_two_streams_and_two_graphs_at_once(dev):
    cases = [case(dev, seed) for seed in (1, 2)]
    want = []
    for run, out in cases:
        run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    streams = [torch.cuda.Stream() for _ in cases]

    def check():
        torch.cuda.synchronize()
        for (_, out), ref in zip(cases, want):
            assert all(torch.equal(a, b) for a, b in zip(out, ref))
            for t in out:
                t.fill_(7.0)
        torch.cuda.synchronize()

    for _ in range(5):
        for (run, _), s in zip(cases, streams):
            with torch.cuda.stream(s):
                run()
        check()
    graphs = []
    for (run, _), s in zip(cases, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            run()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        check()
