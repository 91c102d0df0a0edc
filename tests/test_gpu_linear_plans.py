"""The ways of running a dense product that the sizes of test_gpu_linear and
test_gpu_linear_even leave out, compared bit for bit as there; test_linear_plan
checks on the CPU that between them no kind of plan is left.
"""
import pytest

import test_gpu_linear as linear
import test_gpu_linear_even as even

pytestmark = pytest.mark.gpu

# rows, columns and reduction of the product that is computed, by the widest tile with its last tiles cut
KINDS = [(7032, 3888, 9336), (3880, 4720, 9464), (1304, 7984, 9560), (424, 5968, 9176), (5864, 4464, 5512), (7800, 1072, 5464),
         (2568, 8784, 3384), (4760, 4400, 4200)]
# forwards by the 128 x 128 tile with the deep ring, in parts
FORWARDS = [(3101, 136, 2888), (4622, 200, 2872), (4622, 208, 2872)]


@pytest.mark.parametrize("M,N,K", KINDS)
def test_forward(dev, M, N, K):
    even.test_forward(dev, M, N, K)


@pytest.mark.parametrize("M,N,K", KINDS)
def test_dgrad(dev, M, N, K):
    even.test_dgrad(dev, M, N, K)


@pytest.mark.parametrize("M,N,K", KINDS)
def test_wgrad(dev, M, N, K):
    even.test_wgrad(dev, M, N, K)


@pytest.mark.parametrize("M,N,K", FORWARDS)
def test_forward_in_parts(dev, M, N, K):
    linear.test_forward_exact(dev, M, N, K, linear.F32)
    if N % 16 == 0:                # SwiGLU's columns
        linear.test_forward_exact_in_every_tile(dev, M, N, K)
