"""moe_block_norm on the GPU against its formula in 64 bits."""
from __future__ import annotations

import itertools

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _dense as d
from . import _ops as o

pytestmark = pytest.mark.gpu
EPS = 1e-6


def block(x, gamma, post=None, gate=None, scale=1.0, res=None, res_out=True, y=True, q=True,
          eps=EPS, **kw):
    rows, H = x.shape
    k = dict(device="cuda")
    ro = torch.full((rows, H), 7.0, dtype=torch.bfloat16, **k) if res_out is True else res_out
    oy = torch.full((rows, H), 7.0, dtype=torch.bfloat16, **k) if y is True else y
    oq = torch.full((rows, H), 0xA5, dtype=torch.uint8, **k) if q else None
    os_ = torch.full((rows, H // 128), -1.0, **k) if q else None
    m.moe_block_norm(m.make_shape(1, rows, 1, 1, H), x, gamma, eps, res_out=ro, y=oy, q=oq, s=os_,
                     post_gamma=post, gate=gate, gates=1 if gate is None else gate.shape[0],
                     scale=scale, res=res, **kw)
    torch.cuda.synchronize()
    return ro, oy, oq, os_


def inputs(rows, H, gates=1):
    gen = torch.Generator().manual_seed(rows * 131 + H)

    def t(*shape, by=1.0, plus=0.0):
        return (torch.randn(shape, generator=gen) * by + plus).bfloat16().cuda()
    return (t(rows, H, by=3), t(H, by=0.2, plus=1), t(H, by=0.2, plus=1), t(gates, H, by=0.7),
            t(rows, H))


def check(got, x, gamma, eps=EPS, **kw):
    ro, y, q, s = got
    v, verr, want, yerr = d.block64(x, gamma, eps, **kw)
    if ro is not None:
        o.assert_bf16(ro, v, verr)
    if y is not None:
        o.assert_bf16(y, want, yerr)
    if q is not None:
        o.assert_codes(q, s, want, yerr)


@pytest.mark.parametrize("rows,H", [(1, 128), (1, 7168), (3, 256), (6, 2048), (129, 1408),
                                    (2050, 384), (5, 8192), (2, 65536), (1001, 7168), (3, 8320),
                                    (200, 4224), (330, 8192), (310, 12288), (160, 33024)])
def test_matches_formula(rows, H):
    x, gamma, post, gate, res = inputs(rows, H)
    for kw in (dict(), dict(post=post), dict(post=post, gate=gate, scale=0.5, res=res),
               dict(gate=gate, res=res), dict(res=res, scale=-1.25)):
        check(block(x, gamma, **kw), x, gamma, **kw)


@pytest.mark.parametrize("rows,gates", [(12, 1), (12, 2), (12, 3), (12, 12), (1, 1), (600, 150)])
def test_gate_rows(rows, gates):
    x, gamma, post, gate, res = inputs(rows, 384, gates)
    kw = dict(post=post, gate=gate, res=res, scale=0.22)
    check(block(x, gamma, **kw), x, gamma, **kw)


def test_each_set_of_outputs_is_the_same():
    x, gamma, post, gate, res = inputs(37, 512)
    kw = dict(post=post, gate=gate, res=res)
    full = block(x, gamma, **kw)
    for a, b, c in itertools.product((True, None), (True, None), (True, False)):
        if not (a or b or c):
            continue
        got = block(x, gamma if b or c else None, res_out=a, y=b, q=c, **kw)
        for w, g in zip(full, got):
            assert g is None or torch.equal(w, g)


def test_without_the_first_three_it_is_the_norm():
    """No norm after the branch, no gate, scale 1: moe_rmsnorm, bit for bit."""
    x, gamma, _, _, res = inputs(50, 1024)
    ro, y, q, s = block(x, gamma, res=res)
    r2, y2, q2, s2 = torch.empty_like(ro), torch.empty_like(y), torch.empty_like(q), \
        torch.empty_like(s)
    m.moe_rmsnorm(m.make_shape(1, 50, 1, 1, 1024), x, gamma, EPS, y=y2, q=q2, s=s2, res=res,
                  res_out=r2)
    assert torch.equal(ro, r2)
    o.assert_bf16(y2, *d.block64(x, gamma, EPS, res=res)[2:])
    check((ro, y, q, s), x, gamma, res=res)


@pytest.mark.parametrize("onto", ["x", "res"])
def test_in_place(onto):
    x, gamma, post, gate, res = inputs(33, 2048)
    kw = dict(post=post, gate=gate)
    want = block(x, gamma, res=res, **kw)
    t = dict(x=x.clone(), res=res.clone())
    got = block(t["x"], gamma, res=t["res"], res_out=t[onto], **kw)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    t = dict(x=x.clone(), res=res.clone())
    got = block(t["x"], gamma, res=t["res"], y=t[onto], **kw)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_zero_rows_blocks_and_gamma():
    x = torch.zeros((4, 512), dtype=torch.bfloat16, device="cuda")
    one = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    x[1, 130], x[2] = 2.0, 1.0
    gamma = one.clone()
    gamma[256:384] = 0
    ro, y, q, s = block(x, gamma, post=one)
    for t in (ro, y, q, s):
        assert torch.count_nonzero(t[0]) == 0
    assert s[1].count_nonzero() == 1 and s[1, 1] > 0 and q[1].count_nonzero() == 1
    assert s[2, 2] == 0 and q[2, 256:384].count_nonzero() == 0 and (s[2, [0, 1, 3]] > 0).all()


def test_not_finite_rows_stay_within_their_row():
    x, gamma, post, gate, res = inputs(5, 384)
    kw = dict(post=post, gate=gate, res=res)
    a = block(x, gamma, **kw)
    x[1, 7], res[3, 200] = float("nan"), float("inf")
    b = block(x, gamma, **kw)
    for u, w in zip(a, b):
        assert torch.equal(u[[0, 2, 4]], w[[0, 2, 4]])
    assert b[0][1].isnan().all() and b[1][1].isnan().all() and b[3][1].isnan().all()
    assert (b[2][1] & 0x7F == 0x7F).all()
    assert b[0][3, 200].isinf() and b[0][3].isfinite().sum() == 383
    assert b[1][3, 200].isnan() and b[1][3].count_nonzero() == 1


def test_large_and_tiny_values_and_eps():
    x, gamma, post, gate, res = inputs(2, 256)
    for by, eps in ((1e15, 1e-6), (1e-4, 1e-6), (1e-4, 0.0), (1e-15, 1e-5)):
        a, r = (x.float() * by).bfloat16(), (res.float() * by).bfloat16()
        got = block(a, gamma, gate=gate, res=r, eps=eps)
        v, verr, y, yerr = d.block64(a, gamma, eps, gate=gate, res=r)
        o.assert_bf16(got[0], v, verr + 1e-30)
        o.assert_bf16(got[1], y, yerr + 1e-30)
        o.assert_codes(got[2], got[3], y, yerr + 1e-30)


def test_no_rows_streams_and_graphs():
    e = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    x, gamma, post, gate, res = inputs(300, 256, 3)
    m.moe_block_norm(m.make_shape(1, 0, 1, 1, 256), e, gamma, EPS, y=e, gate=gate, gates=3)
    kw = dict(post=post, gate=gate, res=res, scale=0.5)
    want = block(x, gamma, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = block(x, gamma, stream=side, **kw)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ro, y = torch.zeros_like(x), torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_block_norm(m.make_shape(3, 100, 3, 1, 256), x, gamma, EPS, res_out=ro, y=y,
                         post_gamma=post, gate=gate, gates=3, scale=0.5, res=res)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ro, want[0]) and torch.equal(y, want[1])


def test_offsets_past_32_bits():
    rows, H = 33_000, 65536
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((rows, H), generator=gen, device="cuda", dtype=torch.bfloat16)
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    m.moe_block_norm(m.make_shape(1, rows, 1, 1, H), x, gamma, EPS, y=x, post_gamma=gamma)
    gen.manual_seed(2)
    x0 = torch.randn((rows, H), generator=gen, device="cuda", dtype=torch.bfloat16)
    for at in (slice(0, 2), slice(rows - 2, rows)):
        _, _, y, yerr = d.block64(x0[at], gamma, EPS, post=gamma)
        o.assert_bf16(x[at], y, yerr)
