"""moe_rmsnorm on the GPU against its formula in 64 bits."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _ops as o

pytestmark = pytest.mark.gpu
EPS = 1e-6


def norm64(x, res, gamma, eps=EPS):
    v = x.cpu().double()
    if res is not None:
        v = v + res.cpu().double()
    y = v * (v.square().mean(-1, keepdim=True) + eps).rsqrt() * gamma.cpu().double()
    # the fp32 sum of H squares: at most H additions; the rest is ten operations
    return v, y, (v.shape[-1] / 2 + 10) * o.U * y.abs()


def run(x, gamma, res=None, eps=EPS, y=True, q=True, inplace=False):
    rows, H = x.shape
    sh = m.make_shape(1, rows, 1, 1, H)
    d = dict(device="cuda")
    oy = torch.full((rows, H), 7.0, dtype=torch.bfloat16, **d) if y else None
    oq = torch.full((rows, H), 0xA5, dtype=torch.uint8, **d) if q else None
    os_ = torch.full((rows, H // 128), -1.0, **d) if q else None
    ro = (res if inplace else torch.empty_like(x)) if res is not None else None
    m.moe_rmsnorm(sh, x, gamma, eps, y=oy, q=oq, s=os_, res=res, res_out=ro)
    torch.cuda.synchronize()
    return oy, oq, os_, ro


@pytest.mark.parametrize("rows,H", [(1, 128), (1, 7168), (3, 256), (7, 2048), (129, 1408),
                                    (2049, 384), (5, 8192), (2, 65536), (1001, 7168), (3, 8320)])
@pytest.mark.parametrize("with_res", [False, True])
def test_matches_formula(rows, H, with_res):
    gen = torch.Generator().manual_seed(rows * 131 + H)
    x = o.bf16(torch.randn((rows, H), generator=gen) * 3).cuda()
    res = o.bf16(torch.randn((rows, H), generator=gen)).cuda() if with_res else None
    gamma = o.bf16(1 + 0.2 * torch.randn(H, generator=gen)).cuda()
    v, want, err = norm64(x, res, gamma)
    y, q, s, ro = run(x, gamma, res)
    o.assert_bf16(y, want, err)
    o.assert_codes(q, s, want, err)
    if with_res:
        assert torch.equal(ro.cpu(), (x.cpu().float() + res.cpu().float()).bfloat16())
    # each output alone is the same
    y2, _, _, _ = run(x, gamma, res, q=False)
    _, q2, s2, _ = run(x, gamma, res, y=False)
    assert torch.equal(y, y2) and torch.equal(q, q2) and torch.equal(s, s2)


def test_in_place_residual():
    gen = torch.Generator().manual_seed(5)
    x, res = (o.bf16(torch.randn((33, 2048), generator=gen)).cuda() for _ in range(2))
    gamma = torch.ones(2048, dtype=torch.bfloat16, device="cuda")
    want = (x.float() + res.float()).bfloat16()
    y, _, _, _ = run(x, gamma, res.clone(), q=False)
    y2, _, _, ro = run(x, gamma, res, q=False, inplace=True)
    assert ro is res and torch.equal(ro, want) and torch.equal(y, y2)


def test_zero_rows_blocks_and_gamma():
    x = torch.zeros((4, 512), dtype=torch.bfloat16, device="cuda")
    x[1, 130] = 2.0
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    gamma[256:384] = 0
    x[2] = 1.0
    y, q, s, _ = run(x, gamma)
    assert torch.count_nonzero(y[0]) == 0 and torch.count_nonzero(q[0]) == 0
    assert torch.count_nonzero(s[0]) == 0
    assert s[1].count_nonzero() == 1 and s[1, 1] > 0 and q[1].count_nonzero() == 1
    assert s[2, 2] == 0 and q[2, 256:384].count_nonzero() == 0 and (s[2, [0, 1, 3]] > 0).all()


def test_not_finite_rows_stay_within_their_row():
    gen = torch.Generator().manual_seed(6)
    x = o.bf16(torch.randn((5, 384), generator=gen)).cuda()
    gamma = torch.ones(384, dtype=torch.bfloat16, device="cuda")
    y0, q0, s0, _ = run(x, gamma)
    x[1, 7], x[3, 200] = float("nan"), float("inf")
    y, q, s, _ = run(x, gamma)
    for r in (0, 2, 4):
        assert torch.equal(y[r], y0[r]) and torch.equal(q[r], q0[r]) and torch.equal(s[r], s0[r])
    assert y[1].isnan().all() and s[1].isnan().all()
    assert (q[1] & 0x7F == 0x7F).all()
    # inf * 0: the formula's own NaN, zeros elsewhere
    assert y[3, 200].isnan() and y[3].count_nonzero() == 1


def test_large_and_tiny_values_and_eps():
    gamma = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(8)
    base = torch.randn((2, 256), generator=gen)
    for scale, eps in ((1e15, 1e-6), (1e-4, 1e-6), (1e-4, 0.0), (1e-15, 1e-5)):
        x = o.bf16(base * scale).cuda()
        _, want, err = norm64(x, None, gamma, eps)
        y, q, s, _ = run(x, gamma, eps=eps)
        o.assert_bf16(y, want, err + 1e-30)
        o.assert_codes(q, s, want, err + 1e-30)


def test_empty_and_streams_and_graph():
    gamma = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    m.moe_rmsnorm(m.make_shape(1, 0, 1, 1, 256), torch.empty((0, 256), dtype=torch.bfloat16,
                                                             device="cuda"), gamma, EPS,
                  y=torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"))
    gen = torch.Generator().manual_seed(9)
    x = o.bf16(torch.randn((300, 256), generator=gen)).cuda()
    want, _, _, _ = run(x, gamma, q=False)
    sh, st = m.make_shape(3, 100, 3, 1, 256), torch.cuda.Stream()
    y = torch.zeros_like(x)
    st.wait_stream(torch.cuda.current_stream())
    m.moe_rmsnorm(sh, x, gamma, EPS, y=y, stream=st)
    st.synchronize()
    assert torch.equal(y, want)
    y.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_rmsnorm(sh, x, gamma, EPS, y=y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
