"""GPU tests of every launch that the rules can choose for a layer product and
that no shape of tests/test_linear_gpu.py takes; tests/test_shape_rules_cpu.py
checks that the lists leave none out.  Against tests/linear_ref.py."""
import pytest

from tests.test_linear_gpu import test_backward as check_backward
from tests.test_linear_gpu import test_each_gradient_alone as check_alone
from tests.test_linear_gpu import test_forward as check_forward

pytestmark = pytest.mark.gpu

# Both gradients in one launch of 256-wide tiles, dW's or dx's first; wide tiles
# of a split contraction; rows of few tokens past the cache, whole and split;
# two tokens by the weight's rows.
FORMS = [(606, 513, 6931), (69, 422, 16776), (1089, 795, 5125), (1494, 1209, 5875), (229, 399, 17152),
         (5, 26592, 24), (3297, 3563, 1201), (4036, 2569, 1561), (4425, 2118, 1998), (1079, 3726, 1298),
         (1306, 4251, 1527), (1403, 6920, 1420), (2, 7, 9), (970, 1488, 3735), (1186, 1543, 8416)]
PAST_THE_CACHE = [(13, 16403, 8216), (12, 5200, 26016), (30, 16403, 8216), (30, 5203, 26024)]


@pytest.mark.parametrize("T,N,K", FORMS)
def test_forms(T, N, K):
    check_forward(T, N, K, "none", False, False, False)
    check_forward(T, N, K, "silu", True, True, True)
    check_backward(T, N, K, "gelu_tanh", True)
    check_backward(T, N, K, "none", False)
    check_alone(T, N, K)


@pytest.mark.parametrize("T,N,K", PAST_THE_CACHE)
def test_forward_past_the_cache(T, N, K):
    check_forward(T, N, K, "none", False, False, False)
    check_forward(T, N, K, "silu", True, True, True)
