"""The experts' weighted sum and its gradients on the GPU against the formulas in
64 bits.  A sum of k products and the base is off by at most (k + 1) 2^-24 of its
terms' sizes before it is rounded to bf16; a row's gradient is one product,
rounded once (2^-8) after fp32's (2^-24); a weight's gradient is a tree of H
products at most 48 deep."""
import pytest
import torch

import moe_expert_grouped_gemm_amd as ptm

pytestmark = pytest.mark.gpu

F64, BF16 = torch.float64, torch.bfloat16
U = 2.0 ** -24


def make(dev, T, H, k, seed, spare=3, dropped=0.1):
    g = torch.Generator(device=dev).manual_seed(seed)
    M = T * k + spare                                        # rows that nobody owns
    row_of = torch.randperm(M, generator=g, device=dev)[: T * k].view(T, k)
    row_of = torch.where(torch.rand((T, k), generator=g, device=dev) < dropped, -1, row_of).int().contiguous()
    n = lambda *s: torch.randn(s, generator=g, device=dev)
    return {"rows": n(M, H).to(BF16), "weights": n(T, k), "row_of": row_of, "base": n(T, H).to(BF16), "dout": n(T, H).to(BF16),
            "M": M}


def combine(s, weights=True, base=True, out=None):
    T, k = s["row_of"].shape
    H = s["rows"].shape[1]
    if out is None:
        out = torch.full((T, H), 7.0, dtype=BF16, device=s["rows"].device)
    ptm.pt_moe_combine(s["rows"], s["weights"] if weights else None, s["row_of"], s["base"] if base else None, out, T, s["M"], H, k)
    torch.cuda.synchronize()
    return out


def backward(s, weights=True, drows=True, dweights=True):
    T, k = s["row_of"].shape
    M, H = s["rows"].shape
    dev = s["rows"].device
    dr = torch.full((M, H), 9.0, dtype=BF16, device=dev) if drows else None
    dw = torch.full((T, k), 9.0, device=dev) if dweights else None
    ptm.pt_moe_combine_bwd(s["dout"], s["rows"] if dweights else None, s["weights"] if weights else None, s["row_of"], dr, dw, T,
                           M, H, k)
    torch.cuda.synchronize()
    return dr, dw


def wide(s, weights):
    """Each slot's row [T, k, H] and weight in 64 bits, zeros for a slot without a row."""
    ok = (s["row_of"] >= 0) & (s["row_of"] < s["M"])
    rows = s["rows"][s["row_of"].long().clamp(0, s["M"] - 1)].to(F64) * ok[:, :, None]
    w = s["weights"].to(F64) if weights else torch.ones_like(s["weights"], dtype=F64)
    return ok, rows, w


SHAPES = [(1, 8, 1), (1, 4096, 6), (3, 40, 2), (5, 2880, 4), (7, 512, 16), (70, 1032, 5), (33, 2056, 8), (9, 4104, 3), (4, 8200, 2),
          (3, 16392, 2), (2, 32768, 3), (2000, 264, 4)]


@pytest.mark.parametrize("T,H,k", SHAPES)
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("base", [True, False])
def test_combine(dev, T, H, k, weights, base):
    s = make(dev, T, H, k, T + H + k)
    ok, rows, w = wide(s, weights)
    start = s["base"].to(F64) if base else torch.zeros((T, H), dtype=F64, device=dev)
    want = start + (rows * w[:, :, None]).sum(1)
    off = (k + 1) * U * (start.abs() + (rows * w[:, :, None]).abs().sum(1))
    out = combine(s, weights, base)
    assert ((out.to(F64) - want).abs() <= 2.0 ** -8 * (want.abs() + off) + off).all()
    if base:
        own = s["base"].clone()
        assert torch.equal(combine(dict(s, base=own), weights, True, out=own), out)


@pytest.mark.parametrize("T,H,k", SHAPES)
@pytest.mark.parametrize("weights", [True, False])
def test_backward(dev, T, H, k, weights):
    s = make(dev, T, H, k, T + H + k + 1)
    ok, rows, w = wide(s, weights)
    dr, dw = backward(s, weights)
    dout = s["dout"].to(F64)[:, None, :]
    want = (w[:, :, None] * dout)[ok]
    got = dr[s["row_of"][ok].long()].to(F64)
    assert ((got - want).abs() <= (2.0 ** -8 + 2 * U) * want.abs() + 1e-38).all()
    named = torch.zeros(s["M"], dtype=torch.bool, device=dev)
    named[s["row_of"][ok].long()] = True
    assert (dr[~named] == 9).all()                           # rows that no slot names are left as they were
    prod = rows * dout
    assert ((dw.to(F64) - prod.sum(2)).abs() <= 48 * U * prod.abs().sum(2)).all() and (dw[~ok] == 0).all()
    # each gradient alone has the same bits
    assert torch.equal(backward(s, weights, dweights=False)[0], dr)
    assert torch.equal(backward(s, weights, drows=False)[1], dw)


def test_gather_and_its_gradient(dev):
    """Without weights the backward is the gather of the experts' operand, and the forward its gradient."""
    s = make(dev, 300, 528, 4, 5, spare=0, dropped=0.0)
    dr, _ = backward(s, weights=False, dweights=False)
    assert torch.equal(dr[s["row_of"].long()], s["dout"][:, None, :].expand(-1, 4, -1))
    # <gather(x), r> == <x, combine(r)> for integers
    x, r = torch.randint(-3, 4, (300, 528), device=dev).to(BF16), torch.randint(-3, 4, (1200, 528), device=dev).to(BF16)
    a, _ = backward(dict(s, dout=x), weights=False, dweights=False)
    b = combine(dict(s, rows=r), weights=False, base=False)
    assert (a.to(F64) * r.to(F64)).sum() == (x.to(F64) * b.to(F64)).sum()


def test_slots_out_of_range_nan_and_no_rows(dev):
    s = make(dev, 6, 264, 3, 6, spare=0, dropped=0.0)
    ref, (rdr, rdw) = combine(s), backward(s)
    t = dict(s, row_of=s["row_of"].clone(), weights=s["weights"].clone())
    t["row_of"][0] = torch.tensor([-1, s["M"], 2 ** 31 - 1], device=dev, dtype=torch.int32)   # no rows at all
    t["row_of"][1, 1] = -2 ** 31
    t["weights"][1, 1] = float("nan")                        # the weight of a slot without a row is not read
    out, (dr, dw) = combine(t), backward(t)
    assert torch.equal(out[0], s["base"][0]) and (dw[0] == 0).all() and dw[1, 1] == 0
    assert torch.isfinite(out[1]).all() and torch.equal(out[2:], ref[2:]) and torch.equal(dw[2:], rdw[2:])
    assert (dr[s["row_of"][0].long()] == 9).all()
    # a NaN or an infinity stays in the tokens that read its row
    t = dict(s, rows=s["rows"].clone())
    t["rows"][s["row_of"][4, 0].long(), 7] = float("nan")
    out, (_, dw) = combine(t), backward(t)
    assert torch.isnan(out[4, 7]) and torch.isnan(dw[4, 0]) and torch.isfinite(dw[4, 1:]).all()
    keep = torch.arange(6, device=dev) != 4
    assert torch.equal(out[keep], ref[keep]) and torch.equal(dw[keep], rdw[keep])
    # no rows in the matrix, no tokens
    empty = dict(s, rows=torch.empty((0, 264), dtype=BF16, device=dev), M=0)
    assert torch.equal(combine(empty), s["base"])
    none = {"rows": s["rows"], "weights": s["weights"][:0], "row_of": s["row_of"][:0], "base": s["base"][:0],
            "dout": s["dout"][:0], "M": s["M"]}
    combine(none), backward(none)


def test_far_rows(dev):
    """Rows whose bytes lie past 32 bits."""
    H, M = 32768, 70000                                       # 4.6 GB
    rows = torch.empty((M, H), dtype=BF16, device=dev)
    pick = torch.tensor([[0, M - 1], [65536, 32768]], dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    for r in pick.flatten().tolist():
        rows[r] = torch.randint(-3, 4, (H,), generator=g, device=dev).to(BF16)
    s = {"rows": rows, "weights": torch.tensor([[1.0, 2.0], [4.0, 0.5]], device=dev), "row_of": pick, "M": M,
         "base": torch.zeros((2, H), dtype=BF16, device=dev), "dout": torch.randint(-3, 4, (2, H), generator=g, device=dev).to(BF16)}
    want = (rows[pick.long()].to(F64) * s["weights"].to(F64)[:, :, None])
    assert torch.equal(combine(s), want.sum(1).to(BF16))
    dw = torch.empty((2, 2), device=dev)
    want = (rows[pick.long()].to(F64) * s["dout"].to(F64)[:, None, :]).sum(2)
    ptm.pt_moe_combine_bwd(s["dout"], rows, s["weights"], pick, rows, dw, 2, M, H, 2)
    assert torch.equal(dw, want.float())
    assert torch.equal(rows[pick.long()], (s["weights"][:, :, None] * s["dout"].float()[:, None, :]).to(BF16))


def test_repeats_streams_and_graph(dev):
    s = make(dev, 900, 1056, 6, 9)
    T, k, H, M = 900, 6, 1056, s["M"]
    ref, (rdr, rdw) = combine(s), backward(s)
    out, dr, dw = torch.empty_like(ref), torch.full_like(rdr, 9.0), torch.empty_like(rdw)

    def run():
        ptm.pt_moe_combine(s["rows"], s["weights"], s["row_of"], s["base"], out, T, M, H, k)
        ptm.pt_moe_combine_bwd(s["dout"], s["rows"], s["weights"], s["row_of"], dr, dw, T, M, H, k)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        assert torch.equal(out, ref) and torch.equal(dr, rdr) and torch.equal(dw, rdw)
        out.zero_(), dw.zero_(), dr.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(dr, rdr) and torch.equal(dw, rdw)
