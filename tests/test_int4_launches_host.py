"""Which kernel configurations the 4-bit products launch (no GPU needed)."""
import itertools

import pytest

from tests.int4_cases import DENSE, ROUTED, config


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("pair", [False, True])
def test_every_configuration_has_a_case(group, pair):
    """What the rule chooses over a sweep of sizes, whole and part chunks of K,
    is what the GPU tests' lists run, with a pair map and without one."""
    widths = sorted({int(16 * 1.11 ** i) + d for i in range(82) for d in (0, 1)})
    whole = [640] if group == 128 else [640, 640 + group]
    routed, dense = set(), set()
    for N, K in itertools.product(widths, whole):
        for rows in (1, 2, 3, 4, 5, 6, 8, 9, 16, 17, 24, 32, 33, 64, 200, 1000, 9000):
            dense.add(config(rows, 1, 1, False, N, K, group, pair))
            routed |= {config(rows, E, E, True, N, K, group, pair) for E in (1, 3, 8, 32, 128, 1024)}
    assert len(routed) >= 11 and len(dense) >= 11
    assert routed == {config(T * k, E, E, True, N, K, g, p) for T, k, E, N, K, g, _, p in ROUTED
                      if (g, p) == (group, pair)}
    assert dense == {config(rows, 1, 1, False, N, K, g, p) for rows, N, K, g, _, p in DENSE if (g, p) == (group, pair)}


@pytest.mark.parametrize("rows,E,E_loc", [(1024, 256, 32), (128, 128, 16), (4096, 128, 4), (512, 1024, 128),
                                            (96, 24, 8)])
@pytest.mark.parametrize("pair", [False, True])
def test_a_share_is_taken_for_its_own_rows(rows, E, E_loc, pair):
    """A map over part of the experts launches what a map over those experts
    alone does, with the rows that fall to them."""
    for N, group in itertools.product((64, 1500, 4096, 20000), (32, 64, 128)):
        assert config(rows, E, E_loc, True, N, 1536, group, pair) == \
            config(rows * E_loc // E, E_loc, E_loc, True, N, 1536, group, pair)


@pytest.mark.parametrize("pair", [False, True])
def test_a_share_that_may_hold_every_row_is_not_taken_in_fours(pair):
    """A map of pairs that are all local, over part of the experts."""
    assert config(512, 256, 32, True, 1536, 4096, 128, pair)[2] == 16
    assert config(256, 256, 32, True, 1536, 4096, 128, pair)[2] == 4
