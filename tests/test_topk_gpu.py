"""moe_topk on the GPU against its definition in 64 bits: equal ids, weights within
fp32's error."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _dense as d

pytestmark = pytest.mark.gpu
INF = float("inf")


def choose(logits, R, N=1, **kw):
    rows, E = logits.shape
    idx = torch.full((rows, R), -5, dtype=torch.int32, device="cuda")
    w = torch.full((rows, R), 9.0, device="cuda")
    m.moe_topk(m.make_shape(N, rows // N, E, R, 128), logits.cuda(), idx, w,
               **{k: v.cuda() if torch.is_tensor(v) else v for k, v in kw.items()})
    torch.cuda.synchronize()
    return idx.cpu(), w.cpu()


def check(logits, R, **kw):
    idx, w = choose(logits, R, **kw)
    want, ww = d.topk64(logits, R, **{k: v for k, v in kw.items() if k != "N"})
    assert torch.equal(idx, want), (idx != want).nonzero()[:4]
    d.assert_f32(w, ww, d.topk_error(logits, ww))
    return idx, w


def draw(rows, E, seed, coarse=False):
    gen = torch.Generator().manual_seed(seed)
    l = 1.5 * torch.randn((rows, E), generator=gen)
    return (l.bfloat16().float() if coarse else l), 0.1 * torch.randn(E, generator=gen)


@pytest.mark.parametrize("rows,E,R", [(1, 1, 1), (1, 8, 8), (5, 2, 1), (7, 33, 3), (9, 60, 4),
                                      (33, 64, 6), (130, 128, 8), (17, 129, 32), (65, 160, 6),
                                      (50, 256, 8), (3, 257, 7), (20, 384, 8), (31, 511, 9),
                                      (12, 1000, 32), (40, 1024, 32), (66, 32, 1), (31, 36, 8),
                                      (70, 252, 5), (45, 388, 8), (13, 512, 8), (6, 500, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("coarse", [False, True])
def test_matches_definition(rows, E, R, score, coarse):
    l, bias = draw(rows, E, rows + E, coarse)
    check(l, R, score=score)
    check(l, R, score=score, renorm=False, scale=2.5)
    check(l, R, score=score, bias=bias)
    check(l, R, score=score, bias=bias, renorm=False)


@pytest.mark.parametrize("E,groups,kept,R", [(64, 2, 1, 6), (60, 3, 2, 7), (256, 8, 4, 8),
                                             (256, 32, 5, 8), (160, 8, 3, 6), (1024, 16, 4, 32),
                                             (66, 11, 4, 9), (300, 4, 4, 5), (64, 32, 3, 6),
                                             (384, 4, 2, 8), (512, 16, 5, 7), (384, 12, 4, 3),
                                             (128, 2, 1, 8), (448, 7, 3, 5), (512, 2, 1, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
def test_runs_of_experts(E, groups, kept, R, score, best):
    for coarse in (False, True):
        l, bias = draw(57, E, E + groups, coarse)
        for b in (None, bias):
            check(l, R, score=score, groups=groups, kept=kept, best=best, bias=b)


def test_equal_values_go_to_the_lowest_index():
    l = torch.zeros((3, 40))
    l[1, 5:] = 1.0
    l[2, ::3] = -0.0
    for kw in (dict(), dict(bias=torch.zeros(40)), dict(score="sigmoid", bias=torch.ones(40)),
               dict(groups=5, kept=3, best=2), dict(groups=5, kept=3, best=2, bias=torch.zeros(40))):
        idx, _ = check(l, 9, **kw)
        assert idx[0].tolist() == list(range(9)) and idx[2].tolist() == list(range(9))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_that_fp32_cannot_tell_apart(score):
    """Scores a few 2^-26 apart, and runs' worths: their order is that of 64 bits."""
    gen = torch.Generator().manual_seed(1)
    E = 256
    l = torch.zeros((64, E)) + 0.25
    for i in range(64):
        at = torch.randperm(E, generator=gen)[:40]
        l[i, at] += torch.randint(-3, 4, (40,), generator=gen) * 2.0 ** -24
    bias = torch.randint(-2, 3, (E,), generator=gen) * 2.0 ** -27
    for kw in (dict(), dict(groups=8, kept=3, best=2), dict(groups=8, kept=3, best=1),
               dict(groups=16, kept=2, best=2)):
        check(l, 8, score=score, bias=bias, **kw)
    check(l, 8, score=score, groups=8, kept=3, best=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_a_little_apart(score):
    """Neighbours 2^-20 to 2^-50 apart: below fp32's step, above and below that of the
    fixed point; large biases, which that does not hold; long batches' way as well."""
    gen = torch.Generator().manual_seed(7)
    E, rows = 256, 60
    l = torch.randn((rows, E), generator=gen)
    bias = torch.zeros(E)
    for e in range(0, E, 2):  # twins whose logits differ by a few steps
        step = 2.0 ** -torch.randint(20, 25, (rows,), generator=gen)
        l[:, e + 1] = l[:, e] + torch.randint(-2, 3, (rows,), generator=gen) * step
    for b in (bias, bias + 0.25, bias + 2.0 ** -30 * torch.randn(E, generator=gen), bias + 1e5,
              bias - 40000.0, 1e3 * torch.randn(E, generator=gen)):
        for kw in (dict(), dict(groups=8, kept=4, best=2), dict(groups=8, kept=4, best=1)):
            check(l, 8, score=score, bias=b, **kw)
    check(l, 8, score=score, groups=8, kept=4, best=2)
    many = l.repeat(100, 1)  # the way of long batches: the same answers
    for b in (None, bias + 0.25):
        few = choose(l, 8, score=score, bias=b, groups=8, kept=4, best=2)
        long = choose(many, 8, score=score, bias=b, groups=8, kept=4, best=2)
        for a, c in zip(few, long):
            assert torch.equal(a.repeat(100, 1), c)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_come_last(score):
    l, bias = draw(6, 48, 3)
    l[0, 3:] = -INF          # three left for eight places
    l[1] = -INF              # none
    l[2, ::2] = -INF
    l[3, :47] = -INF
    l[4, 16:32] = -INF       # a run without any
    for kw in (dict(), dict(bias=bias), dict(bias=bias, groups=3, kept=2, best=2),
               dict(groups=3, kept=1, best=2), dict(groups=3, kept=2, best=1), dict(renorm=False)):
        idx, w = check(l, 8, score=score, **kw)
        assert (w[1] == 0).all() and w.isfinite().all()
        assert all(len(set(r)) == 8 and min(r) >= 0 and max(r) < 48 for r in idx.tolist())
    tied = l.clone()
    tied[0, :2] = 1.0
    check(tied, 8, score=score, bias=torch.zeros(48))
    low = torch.full((2, 48), torch.finfo(torch.float32).min)
    low[1, 7] = 0.0
    check(low, 4, score=score)
    check(low, 4, score=score, bias=bias)


def test_bias_of_no_value_takes_an_expert_out():
    l, bias = draw(4, 32, 5)
    bias[4], bias[9] = -INF, float("nan")
    idx, _ = check(l, 6, bias=bias)
    assert not torch.isin(idx, torch.tensor([4, 9])).any()
    idx, _ = choose(l, 32, bias=bias)
    assert (idx[:, 30:] == torch.tensor([4, 9])).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", ["plain", "infinite", "all infinite", "none", "huge"])
def test_long_batches_way(score, bias):
    """Tokens that are repeated until they go eight lanes each: what they get alone, with
    biases that put several experts at one value, out of service or beyond fixed point."""
    l, b = draw(40, 64, 12)
    l[3, 5:] = l[7] = -INF
    l[11, 8], l[13, 9] = float("nan"), INF
    l[17] = 0.5
    if bias == "infinite":
        b[5], b[40], b[41] = INF, INF, INF
    elif bias == "all infinite":
        b[:] = INF
    elif bias == "none":
        b[::2], b[1] = -INF, float("nan")
    elif bias == "huge":
        b[7], b[9], b[11], b[33:35] = 3e38, -3e38, 2e38, 16383.0
    rest = [i for i in range(40) if i not in (11, 13)]
    for kw in (dict(), dict(groups=2, kept=1, best=2), dict(groups=2, kept=1, best=1)):
        few = choose(l, 6, score=score, bias=b, **kw)
        check(l[rest], 6, score=score, bias=b, **kw)
        long = choose(l.repeat(500, 1), 6, score=score, bias=b, **kw)
        for a, c in zip(few, long):
            assert torch.equal(a.repeat(500, 1).view(torch.int32), c.view(torch.int32))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_not_a_number_stays_in_its_row(score, with_bias):
    l, bias = draw(9, 64, 4)
    kw = dict(score=score, bias=bias if with_bias else None)
    i0, w0 = choose(l, 6, **kw)
    l[2, 5], l[6, 9] = float("nan"), INF
    idx, w = choose(l, 6, **kw)
    rest = [0, 1, 3, 4, 5, 7, 8]
    assert torch.equal(idx[rest], i0[rest]) and torch.equal(w[rest], w0[rest])
    assert w[2].isnan().all()
    assert w[6].isnan().all() if score == "softmax" else w[6].isfinite().all()
    assert all(len(set(r)) == 6 and min(r) >= 0 and max(r) < 64 for r in idx.tolist())


def test_large_logits():
    l, bias = draw(11, 100, 6)
    for by in (50.0, 1e4, 1e-4):
        for score in ("softmax", "sigmoid"):
            check(l * by, 5, score=score)
            check(l * by, 5, score=score, bias=bias)
            check(l * by, 5, score=score, bias=bias * 1e3)


def test_many_tokens_ranks_streams_and_graphs():
    l, bias = draw(4003, 256, 8)
    kw = dict(score="sigmoid", bias=bias, groups=8, kept=4, best=2, scale=2.5)
    idx, w = check(l, 8, **kw)
    i2, w2 = choose(l[:4000], 8, N=4, **kw)
    assert torch.equal(idx[:4000], i2) and torch.equal(w[:4000], w2)
    dl, db = l.cuda(), bias.cuda()
    gi, gw = torch.zeros_like(idx).cuda(), torch.zeros_like(w).cuda()
    sh, g = m.make_shape(1, 4003, 256, 8, 128), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_topk(sh, dl, gi, gw, **{**kw, "bias": db})
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gi.cpu(), idx) and torch.equal(gw.cpu(), w)
    side = torch.cuda.Stream()
    gi.zero_()
    side.wait_stream(torch.cuda.current_stream())
    m.moe_topk(sh, dl, gi, gw, stream=side, **{**kw, "bias": db})
    side.synchronize()
    assert torch.equal(gi.cpu(), idx)


def test_no_tokens():
    e = torch.empty(0, device="cuda")
    m.moe_topk(m.make_shape(1, 0, 8, 2, 128), e, e, e)
    torch.cuda.synchronize()
