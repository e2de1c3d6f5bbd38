"""Tiles of the grouped products: every one that a plan has is one that there is a kernel for, and is reached."""
import random

from tests import host


def test_tiles_of_each_layout():
    rng = random.Random(3)
    seen = {0: set(), 1: set()}
    for _ in range(60000):
        G, T, N = (int(2 ** rng.uniform(0, top)) for top in (16, 22, 15))
        for rows in (0, 1):
            seen[rows].add(host.lib().grouped_tile(G, T, N, rows))
    assert seen[0] == {64, 128, 256}  # weights stored as N rows of K
    assert seen[1] == {128, 256}      # read along their other axis


def test_groups_past_the_table_do_not_take_the_tiles_that_need_it():
    for rows in (0, 1):
        assert host.lib().grouped_tile(1024, 1024 * 400, 8192, rows) == 256
        assert host.lib().grouped_tile(1025, 1025 * 400, 8192, rows) != 256
