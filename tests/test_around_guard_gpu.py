"""The 16-bit products, the choice and the block's end write nothing outside their
outputs; from one host thread or from several, on streams of their own."""
from __future__ import annotations

import threading

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _ops as o
from .test_operators_guard_gpu import Guarded

pytestmark = pytest.mark.gpu


def rand(gen, *shape):
    return o.bf16(torch.randn(shape, generator=gen)).cuda()


@pytest.mark.parametrize("rows", [1, 17, 61, 130, 300, 700])
@pytest.mark.parametrize("n,k", [(1, 8), (130, 264), (515, 1032), (2048, 2048)])
def test_products(rows, n, k):
    gen = torch.Generator().manual_seed(rows + n)
    x, w, bias, res = rand(gen, rows, k), rand(gen, 2 * n, k), rand(gen, 2 * n), rand(gen, rows, n)
    sh, g, one = m.make_shape(1, rows, 1, 1, 128), Guarded(), w[:n].contiguous()
    b1 = bias[:n].contiguous()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        m.moe_linear(sh, n, k, x, one, g((rows, n), dtype), bias=b1, res=res, act="gelu",
                     status=status)
    m.moe_linear_glu(sh, n, k, x, w, g((rows, n), torch.bfloat16), bias=bias, status=status)
    g.check()
    assert int(status) == 0


@pytest.mark.parametrize("rows,E,R,groups", [(1, 8, 8, 1), (33, 256, 8, 8), (130, 1000, 32, 4),
                                             (15000, 256, 7, 8), (4099, 60, 3, 1)])
def test_choice(rows, E, R, groups):
    l, g = torch.randn((rows, E), device="cuda"), Guarded()
    for bias in (None, torch.zeros(E, device="cuda")):
        m.moe_topk(m.make_shape(1, rows, E, R, 128), l, g((rows, R), torch.int32),
                   g((rows, R), torch.float32), bias=bias, groups=groups, kept=(groups + 1) // 2,
                   score="sigmoid")
    g.check()


@pytest.mark.parametrize("rows,H", [(1, 128), (3, 7168), (1000, 1408), (400, 256), (400, 512),
                                    (2, 65536), (700, 8320)])
def test_block_norm(rows, H):
    gen, g = torch.Generator().manual_seed(rows), Guarded()
    x, v = rand(gen, rows, H), rand(gen, 3, H)
    for post in (None, v[0]):
        m.moe_block_norm(m.make_shape(1, rows, 1, 1, H), x, v[1], 1e-6,
                         res_out=g((rows, H), torch.bfloat16), y=g((rows, H), torch.bfloat16),
                         q=g((rows, H), torch.uint8), s=g((rows, H // 128), torch.float32),
                         post_gamma=post, gate=v[2], res=x)
    g.check()


def test_host_threads_and_streams_at_once():
    """Four host threads, a stream each, every kind of call: the results of calls made
    alone."""
    gen = torch.Generator().manual_seed(4)
    T, E, R, H, I = 40, 64, 6, 512, 384
    x, res = rand(gen, 300, H), rand(gen, 300, H)
    w13, w2, wr = rand(gen, 2 * I, H) / 16, rand(gen, H, I) / 16, rand(gen, E, H) / 16
    gamma, bias = rand(gen, H), torch.randn(E, generator=gen).cuda() / 10

    def calls(stream, n):
        k = dict(device="cuda")
        got = []
        for rows in (1, T, 300):
            sh = m.make_shape(1, rows, E, R, H)
            h = torch.empty((rows, I), dtype=torch.bfloat16, **k)
            y, ro, z = (torch.empty((rows, H), dtype=torch.bfloat16, **k) for _ in range(3))
            l = torch.empty((rows, E), **k)
            idx, w = torch.empty((rows, R), dtype=torch.int32, **k), torch.empty((rows, R), **k)
            got.append((sh, rows, h, y, ro, z, l, idx, w))
        stream.wait_stream(torch.cuda.default_stream())
        for _ in range(n):
            for sh, rows, h, y, ro, z, l, idx, w in got:
                m.moe_linear(sh, E, H, x, wr, l, stream=stream)
                m.moe_topk(sh, l, idx, w, bias=bias, score="sigmoid", groups=8, kept=4, best=2,
                           stream=stream)
                m.moe_linear_glu(sh, I, H, x, w13, h, stream=stream)
                m.moe_linear(sh, H, I, h, w2, y, res=res, stream=stream)
                m.moe_block_norm(sh, y, gamma, 1e-6, res_out=ro, y=z, post_gamma=gamma, res=res,
                                 stream=stream)
        stream.synchronize()
        return [t for g in got for t in g[2:]]
    want = calls(torch.cuda.Stream(), 1)
    got, errors = {}, []

    def work(i):
        try:
            torch.cuda.set_device(0)
            got[i] = calls(torch.cuda.Stream(), 25)
        except Exception as e:  # reported by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(4):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want))
