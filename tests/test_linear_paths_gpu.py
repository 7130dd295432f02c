"""The 16-bit products by each way of their rule (csrc/linear_plan.h): sizes that go
there, with odd edges; and that different ways agree."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _dense as d
from . import _ops as o
from ._linear_plan import plan, way
from ._plan import sms

pytestmark = pytest.mark.gpu


def run(rows, n, k, pair, f32, act, with_bias, with_res, seed=0):
    gen = torch.Generator().manual_seed(rows + n + k + seed)
    outs = 2 * n if pair else n
    x = torch.randn((rows, k), generator=gen).bfloat16().cuda()
    w = (torch.randn((outs, k), generator=gen) / k ** 0.5).bfloat16().cuda()
    bias = (torch.randn(outs, generator=gen) / 2).bfloat16().cuda() if with_bias else None
    res = torch.randn((rows, n), generator=gen).bfloat16().cuda() if with_res else None
    y = torch.full((rows + 2, n), 7.0, dtype=torch.float32 if f32 else torch.bfloat16,
                   device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sh = m.make_shape(1, rows, 1, 1, 128)
    if pair:
        m.moe_linear_glu(sh, n, k, x, w, y, bias=bias, act=act, status=st)
    else:
        m.moe_linear(sh, n, k, x, w, y, bias=bias, res=res, act=act, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and (y[rows:] == 7).all()
    want, err = d.glu64(x, w, bias, act) if pair else d.linear64(x, w, bias, res, act, f32)
    (d.assert_f32 if f32 else o.assert_bf16)(y[:rows], want, err)


@pytest.mark.parametrize("rows,n,k,pair,f32,want", [
    (7, 19457, 128, False, False, "16"), (1, 1, 8, True, False, "16"),
    (1, 1, 8, False, True, "16"), (13, 7160, 1032, False, False, "16/2"),
    (622, 1, 696, True, False, "16/2"), (595, 1, 720, False, True, "16/2"),
    (9, 4099, 648, False, False, "16/4"), (1, 1, 432, True, False, "16/4"),
    (1, 1, 400, False, True, "16/4"), (16, 1000, 2048, False, False, "16/8"),
    (3, 257, 4104, False, True, "16/8"), (5, 70, 1416, True, False, "16/8"),
    (31, 12292, 520, False, False, "32"), (2611, 1, 8, False, True, "32"),
    (2469, 1, 8, True, False, "32"), (30, 6001, 2056, False, False, "32/2"),
    (1223, 1, 1224, False, True, "32/2"), (1468, 1, 1176, True, False, "32/2"),
    (61, 768, 2048, True, False, "32/4"), (593, 1, 832, False, False, "32/4"),
    (1018, 1, 816, False, True, "32/4"), (190, 250, 3336, False, True, "32/8"),
    (257, 1, 1608, False, False, "32/8"), (260, 1, 1632, True, False, "32/8"),
    (60, 18433, 256, False, False, "64"), (96, 7168, 1032, False, False, "64"),
    (5557, 1, 152, True, False, "64"), (5474, 1, 328, False, True, "64"),
    (61, 7167, 3592, False, False, "64/2"), (2790, 1, 2248, False, True, "64/2"),
    (2463, 1, 2616, True, False, "64/2"), (1559, 1, 3896, False, False, "64/4"),
    (1000, 255, 3592, False, True, "64/4"), (1153, 1, 3928, True, False, "64/4"),
    (897, 1, 6912, False, True, "64/8"), (922, 2, 7792, False, False, "64/8"),
    (481, 1, 7864, True, False, "64/8"), (328, 3383, 288, False, False, "128"),
    (257, 5981, 280, False, True, "128"), (6525, 75, 264, True, False, "128"),
    (127, 7166, 7176, False, False, "128/2"), (5697, 52, 3800, False, True, "128/2"),
    (70, 3547, 3880, True, False, "128/2"), (2536, 1, 5320, False, False, "128/4"),
    (2047, 250, 7176, False, True, "128/4"), (2530, 1, 7096, True, False, "128/4"),
    (129, 40000, 64, False, False, "tiles"), (717, 3565, 1064, False, False, "tiles"),
    (2538, 1426, 8, False, False, "tiles"), (1100, 1032, 520, True, False, "tiles"),
    (9000, 130, 1160, False, True, "tiles"),
    # tiles whose outputs' rows start on 8, 4 and 2 bytes
    (1629, 260, 272, False, False, "tiles"), (1647, 258, 256, False, False, "tiles"),
    (3623, 259, 208, False, False, "tiles"), (1132, 1428, 816, False, True, "tiles"),
    (1404, 2594, 400, False, True, "tiles"), (1931, 1451, 888, False, True, "tiles"),
    (834, 3028, 448, True, False, "tiles"), (854, 3482, 840, True, False, "tiles"),
    (1229, 1883, 1080, True, False, "tiles"),
])
def test_way(rows, n, k, pair, f32, want):
    assert way(plan(rows, n, k, pair, f32, sms())) == want
    for act, bias, res in (("none", False, False), ("silu", True, not pair)):
        run(rows, n, k, pair, f32, act, bias, res)


def test_rows_by_different_ways_agree():
    """The same rows as a few, as more and in tiles: within the products' error."""
    gen = torch.Generator().manual_seed(4)
    n, k = 640, 1288
    x = torch.randn((700, k), generator=gen).bfloat16().cuda()
    w = (torch.randn((n, k), generator=gen) / k ** 0.5).bfloat16().cuda()
    want, err = d.linear64(x, w)
    for rows in (1, 16, 17, 33, 65, 129, 257, 700):
        y = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
        m.moe_linear(m.make_shape(1, rows, 1, 1, 128), n, k, x, w, y)
        o.assert_bf16(y, want[:rows], err[:rows])


def test_shape_of_several_ranks():
    gen = torch.Generator().manual_seed(5)
    x = torch.randn((3, 20, 256), generator=gen).bfloat16().cuda()
    w = torch.randn((100, 256), generator=gen).bfloat16().cuda()
    y, z = (torch.empty((3, 20, 100), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.moe_linear(m.make_shape(3, 20, 6, 2, 256), 100, 256, x, w, y)
    m.moe_linear(m.make_shape(1, 60, 1, 1, 128), 100, 256, x, w, z)
    assert torch.equal(y, z)
