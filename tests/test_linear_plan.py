"""The rule by which a 16-bit product takes its kernel, on the host."""
from __future__ import annotations

import random

import pytest

from ._linear_plan import plan, way

SMS, SMEM = 152, 232448


@pytest.mark.parametrize("rows,n,k,pair,f32,want", [
    (1, 7168, 2048, False, False, "16/2"), (1, 256, 7168, False, True, "16/8"),
    (1, 2048, 7168, True, False, "16/4"), (61, 768, 2048, True, False, "32/4"),
    (100, 7168, 2048, False, False, "64"), (2048, 256, 7168, False, True, "128/4"),
    (509, 7168, 7168, False, False, "tiles"), (200, 2048, 7168, True, False, "128/2"),
    (8191, 7168, 7168, False, False, "tiles"), (8191, 2048, 7168, True, False, "tiles"),
    (16000, 256, 7168, False, True, "tiles"), (1, 129280, 7168, False, False, "16"),
])
def test_ways(rows, n, k, pair, f32, want):
    assert way(plan(rows, n, k, pair, f32, SMS)) == want


def test_what_it_chooses_is_possible():
    rng = random.Random(3)
    for _ in range(4000):
        pair = rng.random() < 0.4
        f32 = not pair and rng.random() < 0.4
        sms = rng.choice((152, 148, 132, 16))
        rows, n = (int(2 ** rng.uniform(0, 20)) for _ in range(2))
        k = 8 * int(2 ** rng.uniform(0, 13))
        p = plan(rows, n, k, pair, f32, sms)
        blocks = (k + 63) // 64
        if p.width:
            assert rows > 128 and p.width % (64 if pair else 32) == 0
            assert p.width <= (128 if f32 else 256) and p.parts == 1
            continue
        stages = (blocks + 1) // 2
        assert p.at in (16, 32, 64, 128) and p.at < 2 * max(rows, 9)
        assert p.parts in (1, 2, 4, 8) and p.parts <= stages
        tiles = -(-n // (64 if pair else 128)) * -(-rows // p.at)
        assert p.parts == 1 or tiles * p.parts <= sms
        stage = 2 * (16384 + p.at * 128)
        apart = max(p.at, 4 * p.parts) * 512 if p.at <= 64 else 0
        assert 1 <= p.stages <= 6 and 1280 + apart + p.stages * stage <= SMEM
        assert apart or p.stages * stage >= p.at * 512
        # an SM's 512 columns of tensor memory last for the CTAs that its shared memory holds
        columns = max(32, p.at * (2 if f32 else 1))
        assert 233472 // (1024 + 1280 + apart + p.stages * stage) * columns <= 512
