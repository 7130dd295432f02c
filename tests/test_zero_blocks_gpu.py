"""A block of 128 whose scale is zero has zero bytes, whatever the signs of its
zeros: as the dispatch codes one."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _ops as o

pytestmark = pytest.mark.gpu
ONE, NEG = 0x38, 0xB8  # 1.0 and -1.0 in e4m3


@pytest.mark.parametrize("H", [256, 65536])
def test_norm(H):
    """Zeros of either sign times a gamma of either sign, and values so small that
    their scale rounds to zero."""
    x = torch.zeros((4, H), dtype=torch.bfloat16, device="cuda")
    x[1] = -0.0
    x[2, ::2], x[2, 1::2] = 2.0 ** -133, -2.0 ** -133
    x[3, :128] = 1.0
    gamma = torch.full((H,), -2.0 ** -14, dtype=torch.bfloat16, device="cuda")
    gamma[::3] = 2.0 ** -14
    q = torch.full((4, H), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((4, H // 128), -1.0, device="cuda")
    m.moe_rmsnorm(m.make_shape(1, 4, 1, 1, H), x, gamma, 1.0, q=q, s=s)
    assert s[:3].count_nonzero() == 0 and q[:3].count_nonzero() == 0
    assert s[3, 0] > 0 and (q[3, :128] & 0x7F == 0x7E).all()
    assert s[3, 1:].count_nonzero() == 0 and q[3, 128:].count_nonzero() == 0


def gates_and_ups(inter, k):
    """Weights whose gates are -k, and whose ups are zero in every second block."""
    q = torch.full((1, 2 * inter, k), NEG, dtype=torch.uint8)
    for b in range(inter // 128):
        q[:, inter + b * 128:inter + (b + 1) * 128] = 0 if b % 2 else ONE
    return q.cuda(), torch.full((1, 2 * inter // 128, k // 128), 1 / 128, device="cuda")


def check(hq, hs, inter):
    hq, hs = hq.view(-1, inter // 128, 128), hs.view(-1, inter // 128)
    assert hs[:, 1::2].count_nonzero() == 0 and hq[:, 1::2].count_nonzero() == 0
    assert (hs[:, ::2] > 0).all() and (hq[:, ::2] == 0xFE).all()


@pytest.mark.parametrize("rows,inter,k", [(3, 256, 128), (300, 1280, 256), (300, 640, 4096)])
def test_products(rows, inter, k):
    """Few rows; tiles; tiles that two CTAs share."""
    d = dict(device="cuda")
    a, a_s = torch.full((rows, k), ONE, dtype=torch.uint8, **d), torch.ones((rows, k // 128), **d)
    a_s /= k // 128
    hq = torch.full((rows, inter), 0xA5, dtype=torch.uint8, **d)
    hs = torch.full((rows, inter // 128), -1.0, **d)
    m.moe_expert_gemm_swiglu(m.make_shape(1, rows, 1, 1, 128, rows), inter, k, a, a_s, None,
                             *gates_and_ups(inter, k), hq, hs)
    check(hq, hs, inter)


@pytest.mark.parametrize("T", [2, 7])
def test_few(T):
    H, inter, d = 256, 256, dict(device="cuda")
    x = torch.full((T, H), 0.5, dtype=torch.bfloat16, **d)
    gen = torch.Generator().manual_seed(T)
    hq = torch.full((T, 1, inter), 0xA5, dtype=torch.uint8, **d)
    hs = torch.full((T, 1, inter // 128), -1.0, **d)
    m.moe_layer_few(m.make_shape(1, T, 1, 1, H), inter, x, torch.zeros((T, 1), dtype=torch.int32, **d),
                    torch.ones((T, 1), **d), *gates_and_ups(inter, H),
                    *(t.cuda() for t in o.make_weights(gen, 1, H, inter)), hq, hs,
                    torch.empty_like(x), torch.zeros(1, dtype=torch.int32, **d))
    check(hq, hs, inter)
