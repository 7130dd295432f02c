"""moe_linear and moe_linear_glu on the GPU against their formulas in 64 bits."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _dense as d
from . import _ops as o

pytestmark = pytest.mark.gpu
ACTS = list(m.MOE_ACTS)


def inputs(rows, n, k, seed=0):
    gen = torch.Generator().manual_seed(seed + 7 * rows + 31 * n + k)

    def t(*shape, by=1.0):
        return (torch.randn(shape, generator=gen) * by).bfloat16().cuda()
    return t(rows, k), t(n, k, by=k ** -0.5), t(n, by=0.5), t(rows, n), t


def linear(x, w, bias=None, res=None, act="none", f32=False, y=None, **kw):
    rows, (n, k) = x.shape[0], w.shape
    if y is None:
        y = torch.full((rows, n), 7.0, dtype=torch.float32 if f32 else torch.bfloat16,
                       device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.moe_linear(m.make_shape(1, rows, 1, 1, 128), n, k, x, w, y, bias=bias, res=res, act=act,
                 status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0
    return y


SIZES = [(1, 1, 8), (1, 128, 64), (2, 3, 16), (3, 129, 72), (15, 127, 120), (16, 256, 256),
         (17, 100, 40), (31, 384, 4096), (33, 260, 1000), (64, 130, 512), (65, 640, 136),
         (127, 66, 264), (128, 128, 1024), (129, 500, 2056), (200, 1028, 328), (255, 256, 64),
         (257, 384, 192), (300, 1000, 520), (513, 258, 1288), (260, 33, 8), (1024, 512, 128),
         (1500, 771, 456), (259, 2570, 3200)]


@pytest.mark.parametrize("rows,n,k", SIZES)
def test_linear_matches_formula(rows, n, k):
    x, w, bias, res, _ = inputs(rows, n, k)
    p = d.linear64(x, w)
    o.assert_bf16(linear(x, w), *p)
    d.assert_f32(linear(x, w, f32=True), *d.linear64(x, w, f32=True))
    act = ACTS[(rows + n + k) % 6]
    o.assert_bf16(linear(x, w, bias, res, act), *d.linear64(x, w, bias, res, act))
    d.assert_f32(linear(x, w, bias, res, act, f32=True), *d.linear64(x, w, bias, res, act, True))


@pytest.mark.parametrize("rows,inter,k", SIZES)
def test_glu_matches_formula(rows, inter, k):
    x, w, bias, _, _ = inputs(rows, 2 * inter, k)
    for b, act in ((None, "silu"), (bias, ACTS[(rows + inter + k) % 6])):
        h = torch.full((rows, inter), 7.0, dtype=torch.bfloat16, device="cuda")
        m.moe_linear_glu(m.make_shape(1, rows, 1, 1, 128), inter, k, x, w, h, bias=b, act=act)
        o.assert_bf16(h, *d.glu64(x, w, b, act))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("f32", [False, True])
def test_activations_over_their_range(act, f32):
    """One product of 1 and v: large, small and middling values of both signs, both
    zeros; infinities and NaN as the formula has them."""
    v = torch.cat([torch.linspace(-30, 30, 601), torch.tensor([0.0, -0.0, 1e-8, -1e-8, 90.0, -90.0,
                                                               3e4, -3e4])]).bfloat16()
    x = torch.zeros((v.numel(), 8), dtype=torch.bfloat16)
    x[:, 0] = v
    w = torch.zeros((16, 8), dtype=torch.bfloat16)
    w[:, 0] = 1
    y = linear(x.cuda(), w.cuda(), act=act, f32=f32)
    want, err = d.linear64(x, w, act=act, f32=f32)
    (d.assert_f32 if f32 else o.assert_bf16)(y, want, err)
    x[0, 0], x[1, 0], x[2, 0] = float("inf"), -float("inf"), float("nan")
    y2 = linear(x.cuda(), w.cuda()[:, :], act=act, f32=f32).cpu()
    assert torch.equal(y2[3:], y.cpu()[3:])
    assert y2[2].isnan().all()
    top = 1.0 if act == "sigmoid" else float("inf")
    assert (y2[0, 0] == top) and (act not in ("relu", "sigmoid") or y2[1, 0] == 0)


def test_rows_see_only_their_own():
    """Infinities and NaN in a row or an output's weights stay there."""
    x, w, _, _, _ = inputs(70, 200, 136)
    y0 = linear(x, w).cpu()
    x2, w2 = x.clone(), w.clone()
    x2[7, 3], x2[69, 135], w2[130, 5] = float("nan"), float("inf"), float("nan")
    y = linear(x2, w2).cpu()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[[7, 69]] = False
    keep[:, 130] = False
    assert torch.equal(y[keep], y0[keep])
    assert y[7].isnan().all() and y[:, 130].isnan().all() and not y[69, :130].isfinite().any()


@pytest.mark.parametrize("rows,n,k", [(3, 130, 264), (33, 512, 2048), (300, 258, 136), (5, 33, 1032),
                                      (100, 1001, 2048), (1629, 260, 272), (1647, 258, 256),
                                      (3623, 259, 208), (1608, 264, 272)])
def test_residual_in_place(rows, n, k):
    x, w, bias, res, _ = inputs(rows, n, k)
    want = linear(x, w, bias, res, "silu")
    y = res.clone()
    assert torch.equal(linear(x, w, bias, y, "silu", y=y), want)


@pytest.mark.parametrize("rows,n,k", [(2, 256, 1024), (40, 1000, 512), (700, 384, 264)])
def test_streams_graphs_and_repeats_agree(rows, n, k):
    x, w, bias, res, _ = inputs(rows, n, k)
    want = linear(x, w, bias, res, "gelu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(linear(x, w, bias, res, "gelu", stream=side), want)
    y = torch.zeros_like(want)
    sh = m.make_shape(1, rows, 1, 1, 128)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_linear(sh, n, k, x, w, y, bias=bias, res=res, act="gelu")
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_calls_follow_each_other_on_a_stream():
    """Each call's input is the call's before it, without a wait on the host.  The gate
    is a sigmoid: x grows by a factor a step (silu would square it until it overflows)."""
    _, w13, b13, _, t = inputs(1, 512, 256)
    w2, x0 = t(256, 256, by=1 / 16), t(24, 256)

    def chain(sync):
        x, h = x0.clone(), torch.empty((24, 256), dtype=torch.bfloat16, device="cuda")
        for _ in range(30):
            m.moe_linear_glu(m.make_shape(1, 24, 1, 1, 128), 256, 256, x, w13, h, bias=b13,
                             act="sigmoid")
            sync()
            m.moe_linear(m.make_shape(1, 24, 1, 1, 128), 256, 256, h, w2, x, res=x)
            sync()
        return x
    want = chain(torch.cuda.synchronize)
    assert want.isfinite().all() and torch.equal(chain(lambda: None), want)


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    m.moe_linear(m.make_shape(1, 0, 1, 1, 128), 8, 64, x, w, x)
    m.moe_linear_glu(m.make_shape(1, 0, 1, 1, 128), 4, 64, x, w, x)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows,n,f32", [(5_000_000, 1, True), (300_001, 8200, False)])
def test_offsets_past_32_bits(rows, n, f32):
    """x of over 2^31 bytes or y of over 2^31 elements: the last rows are right, and the first."""
    k = 256 if n == 1 else 16
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((rows, k), generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.randn((n, k), generator=gen, device="cuda", dtype=torch.bfloat16)
    y = linear(x, w, f32=f32)
    for at in (slice(0, 40), slice(rows // 2, rows // 2 + 40), slice(rows - 40, rows)):
        want = d.linear64(x[at], w, f32=f32)
        (d.assert_f32 if f32 else o.assert_bf16)(y[at], *want)
