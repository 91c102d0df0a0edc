"""A NaN that reaches a gate or an up value of the few-token layer stays a NaN
in the token's output, with and without the clamp of the SwiGLU, whatever the
signs of the weights behind it; the other tokens keep their bits.
"""
import pytest
import torch

from test_gpu_few_tokens import KINDS, make, run

pytestmark = pytest.mark.gpu

NAN = float("nan")


def positive(w, kind):
    """The operand with all its values positive or zero."""
    return w.abs() if kind == "bf16" else w & (0x7F if kind == "mxfp8" else 0x77)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("limit", [0.0, 1.5, 10.0])
def test_nan_in_a_token(dev, kind, limit):
    x, z, _, (a, b) = make(dev, 6, 4, 96, 64, kind, 51)
    for w2 in (b[0], positive(b[0], kind)):
        clean, _, _ = run(x, z, None, a[0], a[1], w2, b[1], 2, 0, 1, 1.0, kind, limit)
        assert clean.isfinite().all()
        bad = x.clone()
        bad[3, 70] = NAN
        out, _, _ = run(bad, z, None, a[0], a[1], w2, b[1], 2, 0, 1, 1.0, kind, limit)
        keep = [0, 1, 2, 4, 5]
        assert out[3].isnan().all() and torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("limit", [0.0, 10.0])
@pytest.mark.parametrize("row", [5, 64 + 9])             # of the gates, of the ups
def test_nan_in_a_weight_row(dev, kind, limit, row):
    x, z, _, (a, b) = make(dev, 5, 4, 96, 64, kind, 53)
    z[:, 3] = float("-inf")
    z[2, 3] = 5.0                                        # the one token of expert 3
    w1, s1, w2 = a[0].clone(), a[1].clone() if a[1] is not None else None, positive(b[0], kind)
    clean, _, _ = run(x, z, None, w1, s1, w2, b[1], 2, 0, 1, 1.0, kind, limit)
    if kind == "bf16":
        w1[3, row, 33] = NAN
    else:
        s1[3, row, 1] = 255                              # E8M0 NaN
    out, _, _ = run(x, z, None, w1, s1, w2, b[1], 2, 0, 1, 1.0, kind, limit)
    keep = [0, 1, 3, 4]
    assert out[2].isnan().all() and torch.equal(out[keep], clean[keep])
