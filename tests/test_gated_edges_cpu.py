"""CPU tests of the gated block's choice of launch, seen through its workspace:
a size that goes by the weights' rows needs none."""
import ctypes

import pytest

from shard_placement_amd import _lib, api
from shard_placement_amd._lib import TideGatedForwardArgs

AT = 1 << 40  # made-up device addresses, far apart


def workspace(T, N, K, x=0, weights=0, ldx=None):
    """Bytes, with x and the weights `x` and `weights` bytes behind an aligned address."""
    a = TideGatedForwardArgs(T, N, K, api.ACTS["silu"], 0, AT + x, ldx or K, 2 * AT + weights, 3 * AT + weights)
    a.h, a.ldh = 4 * AT, N
    n = ctypes.c_size_t(0)
    assert _lib.lib().tide_gated_forward_workspace(ctypes.byref(a), ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("T,N,K", [(2, 14336, 1024), (3, 4096, 512), (3, 13824, 5120), (4, 8192, 2048), (4, 512, 512)])
def test_x_on_any_element_does_not_slow_aligned_weights(T, N, K):
    """Only x is copied, two to four rows of it, before the rings that aligned x takes."""
    copy = -(-2 * T * K // 256) * 256
    aligned = workspace(T, N, K)
    assert workspace(T, N, K, x=2) == aligned + copy
    assert workspace(T, N, K, ldx=K + 1) == aligned + copy
    # weights on any element go by their rows, where they are read in place
    assert workspace(T, N, K, weights=2) == 0


@pytest.mark.parametrize("T,N,K", [(1, 14336, 1024), (2, 13824, 5120), (2, 768, 2048)])
def test_x_on_any_element_by_the_weights_rows(T, N, K):
    assert workspace(T, N, K, x=2) == workspace(T, N, K) == 0
