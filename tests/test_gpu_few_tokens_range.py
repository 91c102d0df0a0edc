"""Weights in 8 and 4 bits at the ends of what their scales can say: values are
taken as bf16, exact from 2^-126 to its largest, in steps of 2^-133 below and
infinite above.  Every weight of FC2 is the same value, so an output is it times
the sum of h, which a value of 1 gives; both are rounded to bf16 once more
(2^-8 each, the fp32 sum of 64 terms 64 * 2^-24).
"""
import pytest
import torch

from test_gpu_few_tokens import make, run

pytestmark = pytest.mark.gpu

ONE = {"mxfp8": 0x38, "mxfp4": 0x22}                     # the codes of 1
CODES = {"mxfp8": {0x01: 2.0 ** -9, 0x08: 2.0 ** -6, 0x38: 1.0, 0x7E: 448.0}, "mxfp4": {0x11: 0.5, 0x22: 1.0, 0x77: 6.0}}


@pytest.mark.parametrize("kind", sorted(CODES))
@pytest.mark.parametrize("size", [1e12, 1.0, 1e-10])     # of x: h goes by its square
def test_ends_of_the_range(dev, kind, size):
    x, z, _, (a, b) = make(dev, 1, 1, 64, 64, kind, 3)
    x = (x.abs() * size).bfloat16()
    w1 = a[0] & (0x7F if kind == "mxfp8" else 0x77)      # all positive: nothing cancels
    scale = torch.full_like(b[1], 127)

    def out(code, byte):
        w2, s = torch.full_like(b[0], code), torch.full_like(b[1], byte)
        return run(x, z, None, w1, a[1], w2, s, 1, 0, 1, 1.0, kind)[0][0, 0].double().item()

    total = out(ONE[kind], 127)
    for code, v in CODES[kind].items():
        for byte in (0, 1, 7, 8, 120, 245, 246, 247, 250, 253, 254):
            value = v * 2.0 ** (byte - 127)
            if value > 3.4e38:
                assert out(code, byte) == float("inf"), (code, byte)
                continue
            want = round(value * 2.0 ** 133) * 2.0 ** -133 * total
            if 2.0 ** -126 < want < 3.3e38 or want == 0:
                assert abs(out(code, byte) - want) <= (2.0 ** -7 + 2.0 ** -15) * want, (code, byte)
