"""The rule by which a product takes its kernel: what it may choose, on the host."""
from __future__ import annotations

import random

import pytest

from ._plan import plan, way

SMS = 152


@pytest.mark.parametrize("N,cap,E,n,k,swiglu,want", [
    (1, 1, 1, 7168, 2048, False, "few"), (1, 32, 1, 7168, 7168, False, "few"),
    (1, 33, 1, 7168, 7168, False, "shared"), (1, 33, 1, 7168, 2048, False, "tiles"),
    (1, 64, 1, 4096, 7168, True, "few"), (1, 128, 1, 4096, 7168, True, "shared"),
    (1, 128, 32, 4096, 7168, True, "few"), (1, 2048, 32, 7168, 2048, False, "tiles"),
    (1, 8191, 1, 7168, 7168, False, "tiles"), (16, 4096, 256, 4096, 7168, True, "tiles"),
])
def test_sizes_go_where_they_are_meant_to(N, cap, E, n, k, swiglu, want):
    assert way(plan(N, cap, E, n, k, swiglu, SMS)) == want


def test_any_plan_has_room_for_any_offsets_and_fits_a_launch():
    rng = random.Random(1)
    seen = set()
    for _ in range(4000):
        N = rng.choice((1, 1, 2, 8))
        E = N * rng.randint(1, 1024 // N)
        cap = int(2 ** rng.uniform(0, 14))
        swiglu = rng.random() < 0.5
        n = 128 * int(2 ** rng.uniform(0, 9)) * (1 + swiglu)
        k = 128 * int(2 ** rng.uniform(0, 9))
        p = plan(N, cap, E, n, k, swiglu, SMS)
        seen.add(way(p))
        at = 16 if p.few else 128
        for _ in range(4):  # cap rows of each rank over its experts, at random
            groups = 0
            for _ in range(N):
                cuts = sorted(rng.randint(0, cap) for _ in range(E // N - 1))
                groups += sum(-(-(b - a) // at) for a, b in zip([0, *cuts], [*cuts, cap]))
            assert groups <= p.units
        nb = n // 128 // (2 if p.few and swiglu else 1)
        assert p.tiles == p.units * -(-nb // p.wide)
        if p.few:
            assert p.units <= 65535 and p.wide == 1  # the grid's second axis
            assert p.parts in (1, 2, 4, 8) and p.parts <= max(1, k // 128)
        else:
            assert p.parts in (1, 2) and p.wide in ((2,) if swiglu else (1, 2))
            assert p.parts == 1 or p.tiles * 2 <= SMS  # a cluster has one tile at most
    assert seen == {"few", "tiles", "shared"}
