"""moe_layer_few calls that follow each other with other rows, ids and weights
each time, over the same scratch: what a kernel read too early would show."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _ops as o

pytestmark = pytest.mark.gpu
STEPS = 12


class Chain:
    """Layers and norms in turn: each layer's rows are the norm of the layer before
    it, and its ids and weights its own."""

    def __init__(self, T, E, R, H, inter, inplace, copied):
        gen = torch.Generator().manual_seed(T * 7 + H)
        self.sh, self.inter = m.make_shape(1, T, E, R, H), inter
        d = dict(device="cuda")
        self.x0 = o.bf16(torch.randn((T, H), generator=gen)).cuda()
        self.idx = [torch.rand((T, E), generator=gen).topk(R, dim=-1).indices.int().cuda()
                    for _ in range(STEPS)]
        self.w = [torch.rand((T, R), generator=gen).cuda() for _ in range(STEPS)]
        self.w13 = [t.cuda() for t in o.make_weights(gen, E, 2 * inter, H)]
        self.w2 = [t.cuda() for t in o.make_weights(gen, E, H, inter)]
        self.gamma = torch.ones(H, dtype=torch.bfloat16, **d)
        self.x = torch.empty_like(self.x0)
        self.out = self.x if inplace else torch.empty_like(self.x0)
        self.hq = torch.empty((T, R, inter), dtype=torch.uint8, **d)
        self.hs = torch.empty((T, R, inter // 128), **d)
        self.status = torch.zeros(1, dtype=torch.int32, **d)
        # ids and weights of every step in the same buffers, or in their own
        self.at = (torch.empty_like(self.idx[0]), torch.empty_like(self.w[0])) if copied else None

    def run(self, sync):
        """Every layer's output."""
        outs = []
        self.x.copy_(self.x0)
        for idx, w in zip(self.idx, self.w):
            if self.at:
                self.at[0].copy_(idx)
                self.at[1].copy_(w)
                idx, w = self.at
            sync()
            m.moe_layer_few(self.sh, self.inter, self.x, idx, w, *self.w13, *self.w2, self.hq,
                            self.hs, self.out, self.status)
            sync()
            if len(outs) % 3 == 2:  # elsewhere kernels of the library follow one another
                outs.append(self.out.clone())
                sync()
            else:
                outs.append(None)
            m.moe_rmsnorm(self.sh, self.out, self.gamma, 1e-6, y=self.x)
            sync()
        return [t for t in [*outs, self.x.clone()] if t is not None]


@pytest.mark.parametrize("copied", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("T,E,R,H,inter", [
    (1, 8, 2, 512, 256), (4, 16, 4, 2048, 768), (5, 16, 4, 2048, 768), (20, 8, 3, 512, 512),
    (64, 32, 8, 1408, 256),
])
def test_calls_with_other_inputs_follow_each_other(T, E, R, H, inter, inplace, copied):
    c = Chain(T, E, R, H, inter, inplace, copied)
    want = c.run(torch.cuda.synchronize)
    assert all(t.isfinite().all() for t in want)
    assert not any(torch.equal(a, b) for a, b in zip(want, want[1:]))
    for _ in range(3):
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


@pytest.mark.parametrize("T,inplace", [(3, False), (3, True), (9, False), (9, True)])
def test_layers_alone_follow_each_other(T, inplace):
    """Nothing between two layers: the first one's output is the second one's rows.
    (A layer without its norm squares small rows, so every second one has it.)"""
    E, R, H, inter = 16, 4, 1024, 512
    c = Chain(T, E, R, H, inter, False, False)
    a, b = c.x, c.x if inplace else c.out

    def run(sync):
        c.x.copy_(c.x0)
        rows, out = a, b
        for i, (idx, w) in enumerate(zip(c.idx, c.w)):
            m.moe_layer_few(c.sh, inter, rows, idx, w, *c.w13, *c.w2, c.hq, c.hs, out, c.status)
            sync()
            rows, out = out, rows
            if i % 2:
                m.moe_rmsnorm(c.sh, rows, c.gamma, 1e-6, y=rows)
                sync()
        return rows.clone()
    want = run(torch.cuda.synchronize)
    assert want.isfinite().all() and want.count_nonzero() > want.numel() // 2
    for _ in range(3):
        assert torch.equal(run(lambda: None), want)
