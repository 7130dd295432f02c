"""Blocks of a few tokens that follow each other without a wait on the host: a router's
product and choice, whose ids and weights the few-token layer takes at once, a shared
expert onto it and the block's end, over the same buffers each time."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _ops as o

pytestmark = pytest.mark.gpu
STEPS = 10


class Chain:
    def __init__(self, T, E, R, H, inter, S, **router):
        gen = torch.Generator().manual_seed(T * 11 + H)

        def t(*shape, by=1.0, plus=0.0):
            return (torch.randn(shape, generator=gen) * by + plus).bfloat16().cuda()
        self.sh, self.dims, self.router = m.make_shape(1, T, E, R, H), (E, H, inter, S), router
        self.x0, self.res0 = t(T, H), t(T, H)
        self.wr, self.s13, self.s2 = t(E, H, by=H ** -0.5), t(2 * S, H, by=H ** -0.5), t(H, S, by=S ** -0.5)
        # a gate and a bias that each step's products make anew
        self.wg, self.wb = t(H, H, by=0.3 * H ** -0.5), t(E, H, by=0.1 * H ** -0.5)
        self.gamma = t(H, by=0.2, plus=1)
        self.w13 = [a.cuda() for a in o.make_weights(gen, E, 2 * inter, H)]
        self.w2 = [a.cuda() for a in o.make_weights(gen, E, H, inter)]
        e = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.x, self.res, self.out, self.both = (e(T, H) for _ in range(4))
        self.logits, self.w, self.idx = e(T, E, dt=torch.float32), e(T, R, dt=torch.float32), \
            e(T, R, dt=torch.int32)
        self.gate, self.bias = e(1, H), e(E, dt=torch.float32)
        self.h, self.hq, self.hs = e(T, S), e(T, R, inter, dt=torch.uint8), \
            e(T, R, inter // 128, dt=torch.float32)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, sync):
        E, H, inter, S = self.dims
        one = m.make_shape(1, 1, E, 1, H)
        self.x.copy_(self.x0)
        self.res.copy_(self.res0)
        got = []
        for step in range(STEPS):
            calls = [
                lambda: m.moe_linear(one, E, H, self.x, self.wb, self.bias),
                lambda: m.moe_linear(self.sh, E, H, self.x, self.wr, self.logits),
                lambda: m.moe_topk(self.sh, self.logits, self.idx, self.w, bias=self.bias,
                                   **self.router),
                lambda: m.moe_layer_few(self.sh, inter, self.x, self.idx, self.w, *self.w13,
                                        *self.w2, self.hq, self.hs, self.out, self.status),
                lambda: m.moe_linear_glu(self.sh, S, H, self.x, self.s13, self.h),
                lambda: m.moe_linear(self.sh, H, S, self.h, self.s2, self.both, res=self.out),
                lambda: m.moe_linear(one, H, H, self.x, self.wg, self.gate, act="sigmoid"),
                lambda: m.moe_block_norm(self.sh, self.both, self.gamma, 1e-6, res_out=self.res,
                                         y=self.x, post_gamma=self.gamma, gate=self.gate,
                                         scale=0.5, res=self.res),
            ]
            for call in calls:
                call()
                sync()
            if step % 4 == 3:  # elsewhere kernels of the library follow one another
                got += [t.clone() for t in (self.x, self.res, self.idx, self.w)]
        return got


@pytest.mark.parametrize("T,E,R,H,inter,S,router", [
    (1, 8, 2, 512, 256, 136, {}), (4, 16, 4, 2048, 256, 512, dict(score="sigmoid")),
    (20, 8, 3, 512, 512, 384, dict(score="sigmoid", groups=4, kept=2, best=2, scale=2.5)),
    (64, 32, 8, 1408, 256, 256, {}),
])
def test_blocks_follow_each_other(T, E, R, H, inter, S, router):
    c = Chain(T, E, R, H, inter, S, **router)
    want = c.run(torch.cuda.synchronize)
    assert all(t.isfinite().all() for t in want) and not torch.equal(want[0], want[4])
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(c.run(lambda: None), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = c.run(lambda: None)
    for _ in range(2):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert int(c.status) == 0
