"""A whole block: norm, router's product and choice, dispatch, experts, combine, shared
expert on top and the block's end, each from what the one before it left, against 64
bits; and as one captured graph."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _dense as d
from . import _ops as o

pytestmark = pytest.mark.gpu
EPS = 1e-6


class Block:
    def __init__(self, N, T, E, R, H, I, S, seed, **router):
        gen = torch.Generator().manual_seed(seed)

        def t(*shape, by=1.0, plus=0.0):
            return (torch.randn(shape, generator=gen) * by + plus).bfloat16().cuda()
        self.shape, self.router = m.make_shape(N, T, E, R, H), router
        self.N, self.T, self.E, self.R, self.H, self.S = N, T, E, R, H, S
        self.res, self.att = t(N, T, H), t(N, T, H)
        self.gamma, self.post, self.after = (t(H, by=0.2, plus=1) for _ in range(3))
        self.gate = t(N, H, by=0.5)
        self.wr, self.s13, self.s2 = t(E, H, by=H ** -0.5), t(2 * S, H, by=H ** -0.5), t(H, S, by=S ** -0.5)
        self.bias = (0.1 * torch.randn(E, generator=gen)).cuda()
        self.w13 = [x.cuda() for x in o.make_weights(gen, E, 2 * I, H)]
        self.w2 = [x.cuda() for x in o.make_weights(gen, E, H, I)]
        self.buf = m.MoeBuffers(N, T, E, R, H)
        e = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.stream, self.x, self.both, self.end, self.nxt = (e(N, T, H) for _ in range(5))
        self.logits, self.w = e(N, T, E, dt=torch.float32), e(N, T, R, dt=torch.float32)
        self.idx, self.h = e(N, T, R, dt=torch.int32), e(N, T, S)
        self.q, self.s = e(N, T, H, dt=torch.uint8), e(N, T, H // 128, dt=torch.float32)

    def run(self, stream=None):
        sh, k = self.shape, dict(stream=stream)
        m.moe_rmsnorm(sh, self.att, self.gamma, EPS, y=self.x, res=self.res, res_out=self.stream, **k)
        m.moe_linear(sh, self.E, self.H, self.x, self.wr, self.logits, **k)
        m.moe_topk(sh, self.logits, self.idx, self.w, bias=self.bias, **self.router, **k)
        self.buf.dispatch(self.x, self.idx, **k)
        self.buf.experts(*self.w13, *self.w2, **k)
        self.buf.combine(self.idx, self.w, **k)
        m.moe_linear_glu(sh, self.S, self.H, self.x, self.s13, self.h, **k)
        m.moe_linear(sh, self.H, self.S, self.h, self.s2, self.both, res=self.buf.out, **k)
        m.moe_block_norm(sh, self.both, self.after, EPS, res_out=self.end, y=self.nxt, q=self.q,
                         s=self.s, post_gamma=self.post, gate=self.gate, gates=self.N, scale=0.5,
                         res=self.stream, **k)

    def outputs(self):
        return [self.x, self.logits, self.idx, self.w, self.buf.out, self.h, self.both, self.end,
                self.nxt, self.q, self.s]


SIZES = [dict(N=2, T=5, E=16, R=4, H=256, I=128, S=136, score="sigmoid", groups=4, kept=2, best=2,
              scale=2.5),
         dict(N=4, T=70, E=64, R=6, H=512, I=256, S=384, score="softmax"),
         dict(N=1, T=1, E=8, R=2, H=1024, I=128, S=512, score="sigmoid")]


@pytest.mark.parametrize("size", range(len(SIZES)))
def test_each_step_from_the_one_before(size):
    b = Block(seed=size, **SIZES[size])
    b.run()
    torch.cuda.synchronize()
    assert int(b.buf.status) == 0
    H, rows = b.H, b.N * b.T
    x = b.x.view(rows, H)
    d.assert_f32(b.logits.view(rows, -1), *d.linear64(x, b.wr, f32=True))
    idx, w = d.topk64(b.logits.view(rows, -1), b.R, bias=b.bias, **b.router)
    assert torch.equal(b.idx.view(rows, b.R).cpu(), idx)
    d.assert_f32(b.w.view(rows, b.R), w, d.topk_error(b.logits, w))
    o.assert_bf16(b.h.view(rows, -1), *d.glu64(x, b.s13))
    out = b.buf.out.view(rows, H)
    o.assert_bf16(b.both.view(rows, H), *d.linear64(b.h.view(rows, -1), b.s2, res=out))
    v, verr, y, yerr = d.block64(b.both.view(rows, H), b.after, EPS, post=b.post, gate=b.gate,
                                 scale=0.5, res=b.stream.view(rows, H))
    o.assert_bf16(b.end.view(rows, H), v, verr)
    o.assert_bf16(b.nxt.view(rows, H), y, yerr)
    o.assert_codes(b.q.view(rows, H), b.s.view(rows, -1), y, yerr)


@pytest.mark.parametrize("size", range(len(SIZES)))
def test_a_graph_and_another_stream_give_the_same(size):
    b = Block(seed=size, **SIZES[size])
    b.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in b.outputs()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run()
    for _ in range(3):
        for t in b.outputs():
            t.view(torch.uint8).zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, b.outputs()))
    side = torch.cuda.Stream()
    for t in b.outputs():
        t.view(torch.uint8).zero_()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        b.run(side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, b.outputs()))


def test_two_blocks_follow_each_other_on_new_inputs():
    """Programmatic launches: the next block's input is this one's end, without a wait
    on the host; the same as with one after every call."""
    size = dict(SIZES[1])
    got = []
    for wait in (False, True):
        b = Block(seed=7, **size)
        for _ in range(6):
            b.run()
            if wait:
                torch.cuda.synchronize()
            b.att.copy_(b.nxt)
            b.res.copy_(b.end)
        torch.cuda.synchronize()
        got.append([t.clone() for t in b.outputs()])
    assert all(torch.equal(a, c) for a, c in zip(*got))
