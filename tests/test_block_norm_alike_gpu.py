"""moe_block_norm without its first three steps, and moe_rmsnorm: two kernels of one
formula.  The residual sums are the same bits.  Their sums of squares are added in other
orders, so that each norm is within (H / 2 + 12) 2^-24 of the formula's (as in _dense) and
the two within (H + 24) 2^-24 of each other, before each is rounded: a bf16 value is
another half step off, 2^-8 at most, a scale 2^-24 and a code half a step of its own."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _dense as d
from . import _ops as o
from .test_block_norm_gpu import EPS, block, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,H", [(1, 128), (50, 1024), (400, 256), (320, 7168), (3, 33024)])
@pytest.mark.parametrize("with_res", [True, False])
def test_block_end_and_norm_agree(rows, H, with_res):
    x, gamma, _, _, res = inputs(rows, H)
    res = res if with_res else None
    ro, y, q, s = block(x, gamma, res=res)
    r2, y2, q2, s2 = (torch.empty_like(t) for t in (ro, y, q, s))
    m.moe_rmsnorm(m.make_shape(1, rows, 1, 1, H), x, gamma, EPS, y=y2, q=q2, s=s2, res=res,
                  res_out=r2)
    torch.cuda.synchronize()
    assert torch.equal(ro, r2)
    near = (H + 24) * 2.0 ** -24
    a, b = y.double(), y2.double()
    assert ((a - b).abs() <= (2 * 2.0 ** -8 + near) * torch.maximum(a.abs(), b.abs())).all()
    a, b = s.double(), s2.double()
    assert ((a - b).abs() <= (2 * 2.0 ** -24 + near) * torch.maximum(a, b) + 2.0 ** -149).all()
    # both codings are the formula's
    want, err = d.block64(x, gamma, EPS, res=res)[2:]
    o.assert_codes(q, s, want, err)
    o.assert_codes(q2, s2, want, err)
    # the same code, or the next one where the two lie on either side of a border
    steps = (code_order(q) - code_order(q2)).abs()
    assert steps.max() <= 1


def code_order(q: torch.Tensor) -> torch.Tensor:
    """The places of e4m3 codes in the order of their values, the two zeros alike."""
    v = q.int()
    return torch.where(v >= 128, 128 - v, v)
