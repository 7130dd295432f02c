"""moe_topk where few experts are in service, tokens are not numbers or biases are as
large as fp32 goes, for short batches (a warp a token) and long ones (eight lanes)."""
from __future__ import annotations

import pytest
import torch

from . import _dense as d
from .test_topk_gpu import INF, check, choose, draw

pytestmark = pytest.mark.gpu
NAN, LEAST = float("nan"), torch.finfo(torch.float32).min
LONG = 15000  # rows that go eight lanes each, with a bias as well


def both_ways(l, R, **kw):
    """The answer for l's rows, which long batches of them get too."""
    idx, w = check(l, R, **kw)
    times = -(-LONG // l.shape[0])
    many = choose(l.repeat(times, 1), R, **kw)
    for a, b in zip((idx, w), many):
        assert torch.equal(a.repeat(times, 1).view(torch.int32), b.view(torch.int32))
    return idx, w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("off", [NAN, -INF])
def test_a_bias_that_takes_an_expert_out_leaves_it_no_weight(score, renorm, off):
    """Fewer experts in service than places: the others fill them, by their index, with
    weight 0, and take nothing from those in service."""
    l, bias = draw(40, 64, 21)
    bias[5:] = off
    bias[3] = -INF
    l[7, 0] = l[8, :5] = -INF
    for kw in (dict(), dict(scale=2.5), dict(groups=2, kept=1, best=1)):
        idx, w = both_ways(l, 8, score=score, renorm=renorm, bias=bias, **kw)
        out = (idx == 3) | (idx > 4) | (torch.gather(l, 1, idx.long()) == -INF)
        assert (out.sum(-1) >= 4).all() and (w[out] == 0).all() and w.isfinite().all()
        if renorm:
            some = (~out).any(-1)
            total = w.double().sum(-1)[some] / kw.get("scale", 1.0)
            assert some.sum() == 39 and (total - 1).abs().max() < 8 * 2.0 ** -23
    l, bias = draw(3, 32, 5)  # all experts are chosen
    bias[4], bias[9] = -INF, NAN
    idx, w = check(l, 32, score=score, renorm=renorm, bias=bias)
    assert (idx[:, 30:] == torch.tensor([4, 9])).all() and (w[:, 30:] == 0).all()
    assert (w[:, :30] > 0).all()


def test_no_expert_in_service():
    l, bias = draw(5, 32, 6)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx, w = choose(l, 4, score=score, renorm=renorm, bias=torch.full((32,), NAN))
            assert (idx == torch.arange(4)).all() and (w == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,R", [(64, 6), (257, 8), (1000, 32)])
def test_not_a_number_gets_different_experts(score, E, R):
    """A token that is not a number has ids that differ, whatever the biases: equal ones
    send it to where near values are ordered again."""
    l, b = draw(9, E, 31)
    l[2, 5], l[6, 9], l[7] = NAN, INF, NAN
    for bias in (torch.zeros(E), torch.full((E,), 0.25), 2.0 ** -24 * b):
        for rows in (9, LONG):
            many = l.repeat(-(-rows // 9), 1)
            idx, w = choose(many, R, score=score, bias=bias)
            s = idx.sort(-1).values
            assert (s[:, 1:] > s[:, :-1]).all() and s.min() >= 0 and s.max() < E
            assert w[2::9].isnan().all() and w[7::9].isnan().all()
            rest = [0, 1, 3, 4, 5, 8]
            want, ww = d.topk64(l[rest], R, score=score, bias=bias)
            assert torch.equal(idx[rest], want)
            d.assert_f32(w[rest], ww, d.topk_error(l[rest], ww))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_runs_whose_worth_is_past_fp32(score):
    """Two values of a run that are finite in fp32, whose sum is not: c is compared in 64
    bits."""
    l, _ = draw(23, 128, 41)
    high = torch.zeros(128)
    high[3], high[5], high[40], high[41], high[70], high[71] = 2e38, 2e38, 3e38, 3e38, 3e38, 2.9e38
    low = torch.zeros(128)
    low[:32], low[32:64], low[64:96], low[96:124] = -INF, LEAST, -3e38, -INF
    part = torch.full((128,), LEAST)
    part[::2] = -3.2e38
    for bias in (high, low, part, -high, torch.full((128,), LEAST)):
        for kept in (1, 2, 3):
            both_ways(l, 8, score=score, bias=bias, groups=4, kept=kept, best=2)
    for bias, kept in ((low, 2), (low, 3), (part, 1)):
        check(l, 30, score=score, bias=bias, groups=4, kept=kept, best=2)
        check(l[:, :120], 17, score=score, bias=bias[:120], groups=5, kept=kept, best=2)  # runs of 24
