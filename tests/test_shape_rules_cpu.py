"""CPU tests of the rules that choose a layer product's tile, split and launch
(tests/shape_rules.py builds them): what every choice has to satisfy."""
import random

import pytest

from tests import shape_rules as rules

CUS = 256


def drawn(n, seed):
    rng = random.Random(seed)
    size = lambda lo, hi: min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))  # noqa: E731
    return [(rng.randrange(3), size(1, 30000), size(1, 30000), size(1, 30000)) for _ in range(n)]


def test_every_choice_covers_the_product():
    """All tiles and all splits that are launched have work, and together they
    cover the outputs and the contraction; a split is a whole number of steps
    of every tile, even for two sets of waves."""
    for kind, I, J, depth in drawn(3000, 1) + [(0, 1 << 22, 2048, 8), (2, 1, 1 << 22, 1 << 11), (1, 8, 1 << 30, 8)]:
        s, us = rules.choose(kind, I, J, depth)
        assert (s.tiles_i - 1) * s.bi < I <= s.tiles_i * s.bi
        assert (s.tiles_j - 1) * s.bj < J <= s.tiles_j * s.bj
        assert (s.splits - 1) * s.split_depth < depth <= s.splits * s.split_depth
        assert s.split_depth % 256 == 0 and s.bk in (64, 256) and s.halves in (1, 2)
        assert us > 0 or J <= 64


def test_few_tokens_go_by_the_weights_rows():
    assert rules.forward(1, 28672, 8192) is None and rules.forward(4, 9, 8) is None
    assert rules.forward(5, 28672, 8192) is not None
    assert rules.forward(1, 28672, 8192, keep=True) is not None
    assert rules.forward(1, 8, 7) is not None


@pytest.mark.parametrize("T,N,K", [(77, 768, 2048), (2048, 13824, 5120), (8, 5120, 5120), (300, 1024, 1024)])
def test_one_gradient_alone_is_no_pair(T, N, K):
    for dx, dw in ((True, False), (False, True), (False, False)):
        assert not rules.gradients(T, N, K, dx, dw)[2]
