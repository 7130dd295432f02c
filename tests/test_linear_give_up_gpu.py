"""What the 16-bit products leave when bounded waits run out: MOE_ST_TIMEOUT, and no
output that those waits were for (as test_give_up_gpu.py: the library compiled once more
with the waits of the second CTA of each cluster's z, or of the second along x, giving up
at once; nothing waits more than a second or two, and nothing faults)."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _dense as d
from . import _ops as o
from ._linear_plan import plan, way
from ._plan import sms
from .test_give_up_gpu import giving_up, path  # noqa: F401

pytestmark = pytest.mark.gpu


def product(rows, n, k, pair=False, f32=False, status=True):
    gen = torch.Generator().manual_seed(rows + n + k)
    x = torch.randn((rows, k), generator=gen).bfloat16().cuda()
    w = (torch.randn((2 * n if pair else n, k), generator=gen) / k ** 0.5).bfloat16().cuda()
    y = torch.full((rows, n), -7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sh = m.make_shape(1, rows, 1, 1, 128)
    kw = dict(status=st if status else None)
    if pair:
        m.moe_linear_glu(sh, n, k, x, w, y, **kw)
    else:
        m.moe_linear(sh, n, k, x, w, y, **kw)
    torch.cuda.synchronize()
    want = d.glu64(x, w) if pair else d.linear64(x, w, f32=f32)
    return y.cpu(), int(st), want


@pytest.mark.parametrize("rows,n,k,pair,f32,want", [
    (16, 1000, 2048, False, False, "16/8"), (61, 768, 2048, True, False, "32/4"),
    (61, 7167, 3592, False, False, "64/2"), (1000, 255, 3592, False, True, "64/4"),
    (200, 2048, 7168, True, False, "128/2"),
])
@pytest.mark.parametrize("status", [True, False])
def test_no_part_of_a_cluster_stores(giving_up, rows, n, k, pair, f32, want, status):  # noqa: F811
    assert way(plan(rows, n, k, pair, f32, sms())) == want
    y, st, _ = product(rows, n, k, pair, f32, status)
    assert (y == -7.0).all()
    assert st == (m.MOE_ST_TIMEOUT if status else 0)


@pytest.mark.parametrize("f32", [False, True])
def test_others_store_theirs(giving_up, f32):  # noqa: F811
    """Few rows, no clusters: the second CTA's 64 rows are not there, the others are."""
    rows, n, k = (5474, 1, 328) if f32 else (150, 18433, 64)
    p = plan(rows, n, k, False, f32, sms())
    assert not p.width and p.parts == 1
    y, st, (want, err) = product(rows, n, k, False, f32)
    lost = slice(p.at, 2 * p.at)
    assert st == m.MOE_ST_TIMEOUT and (y[lost] == -7.0).all()
    kept = torch.ones_like(y, dtype=torch.bool)
    kept[lost] = False
    (d.assert_f32 if f32 else o.assert_bf16)(y[kept], want[kept], err[kept])


def test_a_pairs_second_cta(giving_up):  # noqa: F811
    """Tiles: the first pair's second CTA brings no block beyond its ring, so the pair's
    products end; whatever is stored is right."""
    rows, n, k = 717, 3565, 1064
    assert way(plan(rows, n, k, False, False, sms())) == "tiles"
    y, st, (want, err) = product(rows, n, k)
    assert st == m.MOE_ST_TIMEOUT
    kept = y != -7.0
    assert (~kept).any() and kept.any()
    o.assert_bf16(y[kept], want[kept], err[kept])


def test_the_next_call_is_right(path):  # noqa: F811
    sizes = [(16, 1000, 2048, False), (200, 2048, 7168, True), (717, 3565, 1064, False)]
    with pytest.MonkeyPatch.context() as mp:
        m.lib()
        mp.setattr(m, "_LIB_PATH", path)
        mp.setattr(m, "_lib", None)
        m.lib()
        for size in sizes:
            assert product(*size)[1] == m.MOE_ST_TIMEOUT
    for size in sizes:
        y, st, (want, err) = product(*size)
        assert st == 0
        o.assert_bf16(y, want, err)
