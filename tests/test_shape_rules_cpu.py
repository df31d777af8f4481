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
    """One token, weights that tiles would copy, and, up to four tokens, those
    whose bytes hide the arithmetic; kept z and short rows go by tiles."""
    by_rows = lambda *a, **kw: rules.forward(*a, **kw) is None  # noqa: E731
    assert all(by_rows(1, N, K) for N in (1, 64, 28672) for K in (8, 512, 28672))
    assert all(by_rows(T, 64, 1001) for T in (1, 2, 3, 4))
    assert by_rows(2, 512, 8192) and by_rows(2, 64, 1024) and by_rows(4, 28672, 4096)
    for case in ((2, 256, 512), (2, 256, 8192), (3, 1024, 8192), (4, 4096, 4096), (4, 256, 28672),
                 (5, 28672, 8192), (5, 64, 1001), (1, 8, 7)):
        assert not by_rows(*case), case
    assert not by_rows(1, 28672, 8192, keep=True)


@pytest.mark.parametrize("T,N,K", [(77, 768, 2048), (2048, 13824, 5120), (8, 5120, 5120), (300, 1024, 1024)])
def test_one_gradient_alone_is_no_pair(T, N, K):
    for dx, dw in ((True, False), (False, True), (False, False)):
        assert not rules.gradients(T, N, K, dx, dw)[2]


@pytest.mark.parametrize("tile", range(5))
def test_estimates_count_the_steps_that_run(tile):
    """A contraction that ends inside its split has fewer steps than the split;
    whole splits have all of theirs."""
    us = {d: rules.estimate(rules.GRAD_INPUT, tile, 512, 512, d, 1)[1] for d in (64, 65, 128, 129, 256, 257, 320, 512)}
    pair = rules.estimate(rules.GRAD_INPUT, tile, 512, 512, 64, 1)[0].halves  # two sets of waves take two steps at once
    step = (us[512] - us[256]) / 4
    for d, v in us.items():
        steps = -(-d // (64 * pair)) * pair
        assert abs(v - (us[512] - (8 - steps) * step)) < 1e-9, (d, v)


def test_the_longer_tiles_of_a_joint_launch_come_first():
    """dx's tiles run ceil(N / 64) steps and dW's ceil(T / 64): with tiles of one
    kind the longer contraction is first, also where both round up to the same
    split."""
    seen = set()
    for T in range(1400, 2400, 47):
        for N, K in ((T - 120, 9000), (T + 100, 9000), (T // 2, 12000)):
            x, w, pair, first = rules.gradients(T, N, K)
            if pair and x.bi == 256 and x.bj == w.bj:
                assert first == (-(-N // 64) >= -(-T // 64)), (T, N, K)
                seen.add((first, x.split_depth == w.split_depth))
    assert len(seen) >= 2, seen


@pytest.mark.parametrize("tile", range(5))
def test_wide_tiles_of_dw_pay_for_widening_x(tile):
    """Tiles of 256 columns read x widened in a launch before them; the others
    widen it on the way."""
    s, dx = rules.estimate(rules.GRAD_INPUT, tile, 5120, 4096, 2048, 1)
    _, dw = rules.estimate(rules.GRAD_WEIGHT, tile, 5120, 4096, 2048, 1)
    assert abs(dw - dx - (4 + 3 * 5120 * 2048 / 5.5e6 if s.bi == 256 else 0)) < 1e-9


def test_no_split_is_passed_over():
    """The choice is the least estimate of every tile with every number of splits
    up to 16 that the contraction divides into."""
    off = []
    for kind, I, J, depth in drawn(2500, 2):
        if J <= 64:
            continue
        _, us = rules.choose(kind, I, J, depth)
        for tile in range(rules.lib().tiles()):
            for splits in range(1, 17):
                s, est = rules.estimate(kind, tile, I, J, depth, splits)
                if s.tiles_i * s.tiles_j >= 4 * CUS and splits > 1:
                    break  # tiles enough without
                if est < us * (1 - 1e-9):
                    off.append((kind, I, J, depth, s, est, us))
    assert not off, off[:3]


@pytest.mark.parametrize("I,J,depth,splits", [(768, 77, 8192, 16), (1024, 128, 5120, 10), (81, 493, 3904, 16)])
def test_few_tiles_are_split_far(I, J, depth, splits):
    """Splits that lie behind a number that the contraction does not divide into."""
    assert rules.choose(rules.FORWARD, I, J, rules.round8(depth))[0].splits == splits


@pytest.mark.parametrize("T,N,K,splits", [(94, 2560, 2248, 5), (212, 2560, 912, 5), (1027, 19840, 242, 10)])
def test_dx_gives_up_splits_for_a_joint_launch(T, N, K, splits):
    x, w, pair, _ = rules.gradients(T, N, K)
    assert pair and x.splits == splits and w.splits == 1
    assert rules.choose(rules.GRAD_INPUT, K, T, rules.round8(N))[0].splits > splits


@pytest.mark.parametrize("kind", [rules.FORWARD, rules.GRAD_INPUT, rules.GRAD_WEIGHT])
def test_narrow_tiles_take_two_sets_of_waves_before_two_splits(kind):
    """Up to 2048 elements of contraction where the rule would split in two; above
    it splits, and more than two splits stay splits."""
    for depth, splits, halves in ((512, 1, 1), (520, 1, 2), (1024, 1, 2), (1032, 1, 2), (2048, 1, 2),
                                  (2056, 2, 1), (4096, 2, 1)):
        for J in (17, 40, 64):
            s, _ = rules.choose(kind, 28672, J, depth)
            assert (s.splits, s.halves) == (splits, halves), (depth, J, s)
    assert rules.choose(kind, 28672, 16, 1032)[0].splits == 2  # its tiles have one set
    assert rules.choose(kind, 5120, 40, 1280)[0].splits == 5
    assert rules.choose(kind, 65536, 40, 1024)[0].halves == 1


def test_every_launch_is_tested():
    """No launch that random sizes take is missing from the GPU tests' lists."""
    from tests.test_linear_forms_gpu import FORMS, PAST_THE_CACHE
    from tests.test_linear_gpu import PAIRS, PRODUCTS, TILES

    covered = set().union(*(rules.forms(*s) for s in TILES + PAIRS + PRODUCTS + FORMS))
    covered |= {f for s in PAST_THE_CACHE for f in rules.forms(*s) if f[0] == "forward"}
    rng = random.Random(7)
    size = lambda hi: int(round(hi ** rng.random()))  # noqa: E731
    missing = {}
    for _ in range(60000):
        s = (size(16384), size(30000), size(30000))
        for f in rules.forms(*s) - covered:
            missing.setdefault(f, s)
    assert not missing, missing
    # both gradients in one launch of 256-wide tiles: each width of each, each order
    assert {("both, wide", a, b, c) for a in (192, 256) for b in (192, 256)
            for c in ("dx first", "dW first")} <= covered


def test_grids_fit_at_the_limits():
    """A grid's threads are counted in 32 bits: with the most tokens, features and
    elements a product may have, every choice's grid fits."""
    elements = 1 << 33
    for kind in range(3):
        for I in [1 << k for k in range(0, 23)] + [3, 100, 129, (1 << 22) - 1]:
            for J in [1 << k for k in range(0, 31)] + [(1 << 30) - 1]:
                if kind == rules.GRAD_WEIGHT and J > 1 << 22 or I * J > elements:
                    continue
                for depth in (8, 64, 4096, 1 << 22):
                    if max(I, J) * depth > elements:
                        continue
                    s, _ = rules.choose(kind, I, J, depth)
                    threads = 512 if s.bi == 256 else 256 * s.halves
                    assert s.tiles_i * s.tiles_j * s.splits * threads < 1 << 32, (kind, I, J, depth, s)
                    if s.splits > 1:  # the join's
                        pitch = -(-I // 32) * 32
                        assert J * pitch // 8 < 1 << 32, (kind, I, J, depth, s)
