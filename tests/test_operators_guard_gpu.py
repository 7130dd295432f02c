"""The norm, the products and the few-token layer write nothing outside their
outputs, on one stream or on several, from one host thread or from several."""
from __future__ import annotations

import threading

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _ops as o

pytestmark = pytest.mark.gpu
BAND = 64 * 1024


class Guarded:
    """Device buffers with a band of a known pattern on both sides."""

    def __init__(self):
        self.raw = []

    def __call__(self, shape, dtype):
        n = torch.empty(shape, dtype=dtype, device="meta")
        n = n.numel() * n.element_size()
        raw = torch.full((BAND + n + BAND,), 0x5C, dtype=torch.uint8, device="cuda")
        self.raw.append((raw, n))
        return raw[BAND:BAND + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for raw, n in self.raw:
            assert (raw[:BAND] == 0x5C).all() and (raw[BAND + n:] == 0x5C).all()


@pytest.mark.parametrize("rows,H", [(1, 128), (3, 7168), (200, 1408), (2, 65536)])
def test_norm(rows, H):
    g = Guarded()
    x = o.bf16(torch.randn(rows, H)).cuda()
    m.moe_rmsnorm(m.make_shape(1, rows, 1, 1, H), x, x[0].contiguous(), 1e-6,
                  y=g((rows, H), torch.bfloat16), q=g((rows, H), torch.uint8),
                  s=g((rows, H // 128), torch.float32), res=x,
                  res_out=g((rows, H), torch.bfloat16))
    g.check()


@pytest.mark.parametrize("sizes", [[1], [5, 0, 9], [17], [127, 0, 130], [1] * 40, [400]])
@pytest.mark.parametrize("n,k", [(128, 128), (384, 640), (768, 4096)])
def test_products(sizes, n, k):
    gen = torch.Generator().manual_seed(len(sizes) + n)
    E, rows = len(sizes), sum(sizes)
    off = torch.tensor([[0] + sizes], dtype=torch.int32).cumsum(1).int().cuda()
    a = [t.cuda() for t in o.make_rows(gen, rows, k)]
    w = [t.cuda() for t in o.make_weights(gen, E, 2 * n, k)]
    sh, g = m.make_shape(1, rows, E, 1, 128, rows), Guarded()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.moe_expert_gemm(sh, 2 * n, k, *a, off, *w, g((rows, 2 * n), torch.bfloat16), status)
    m.moe_expert_gemm_swiglu(sh, n, k, *a, off, *w, g((rows, n), torch.uint8),
                             g((rows, n // 128), torch.float32), status)
    g.check()
    assert int(status) == 0


@pytest.mark.parametrize("rows,n,k", [(512, 128, 4096), (512, 512, 256), (9, 128, 1024)])
def test_offsets_that_do_not_ascend(rows, n, k):
    """Rows named twice are more tiles than rows are: the calls end, inside their
    outputs, and the next one is right."""
    gen = torch.Generator().manual_seed(rows + n)
    off = torch.tensor([[0, rows, 0, rows, 0]], dtype=torch.int32).cuda()
    a = [t.cuda() for t in o.make_rows(gen, rows, k)]
    w = [t.cuda() for t in o.make_weights(gen, 4, 2 * n, k)]
    sh, g = m.make_shape(1, rows, 4, 1, 128, rows), Guarded()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, hq = g((rows, n), torch.bfloat16), g((rows, n), torch.uint8)
    hs = g((rows, n // 128), torch.float32)
    m.moe_expert_gemm(sh, n, k, *a, off, w[0][:, :n].contiguous(), w[1][:, :n // 128].contiguous(),
                      y, status)
    m.moe_expert_gemm_swiglu(sh, n, k, *a, off, *w, hq, hs, status)
    g.check()
    assert int(status) == 0
    off = torch.tensor([[0, rows, rows, rows, rows]], dtype=torch.int32).cuda()
    m.moe_expert_gemm_swiglu(sh, n, k, *a, off, *w, hq, hs, status)
    torch.cuda.synchronize()
    p, err = o.product64(a[0].cpu(), a[1].cpu(), w[0][0].cpu(), w[1][0].cpu())
    o.assert_codes(hq.cpu(), hs.cpu(), *o.swiglu64(p, err))


@pytest.mark.parametrize("T,E,R,H,I", [(1, 8, 2, 128, 128), (5, 16, 4, 1408, 256),
                                       (33, 4, 2, 256, 384), (64, 32, 8, 512, 128)])
def test_few(T, E, R, H, I):
    gen = torch.Generator().manual_seed(T)
    idx = torch.rand((T, E), generator=gen).topk(R, dim=-1).indices.int().cuda()
    w = torch.rand((T, R), generator=gen).cuda()
    w13 = [t.cuda() for t in o.make_weights(gen, E, 2 * I, H)]
    w2 = [t.cuda() for t in o.make_weights(gen, E, H, I)]
    x, g = o.bf16(torch.randn((T, H), generator=gen)).cuda(), Guarded()
    m.moe_layer_few(m.make_shape(1, T, E, R, H), I, x, idx, w, *w13, *w2,
                    g((T, R, I), torch.uint8), g((T, R, I // 128), torch.float32),
                    g((T, H), torch.bfloat16), g((1,), torch.int32))
    g.check()


def test_host_threads_and_streams_at_once():
    """Four host threads, a stream each, every kind of call: the results of calls
    made alone."""
    gen = torch.Generator().manual_seed(4)
    T, E, R, H, I = 6, 16, 4, 512, 256
    idx = torch.rand((T, E), generator=gen).topk(R, dim=-1).indices.int().cuda()
    w = torch.rand((T, R), generator=gen).cuda()
    w13 = [t.cuda() for t in o.make_weights(gen, E, 2 * I, H)]
    w2 = [t.cuda() for t in o.make_weights(gen, E, H, I)]
    x = o.bf16(torch.randn((T, H), generator=gen)).cuda()
    rows = [200, 12]
    coded = [[t.cuda() for t in o.make_rows(gen, r, H)] for r in rows]
    offs = [torch.linspace(0, r, E + 1).int()[None].cuda() for r in rows]

    def calls(stream, n):
        out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        hq = torch.empty((T, R, I), dtype=torch.uint8, device="cuda")
        hs = torch.empty((T, R, I // 128), device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        qs = [torch.empty((r, I), dtype=torch.uint8, device="cuda") for r in rows]
        ss = [torch.empty((r, I // 128), device="cuda") for r in rows]
        y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        stream.wait_stream(torch.cuda.default_stream())
        for _ in range(n):
            m.moe_layer_few(m.make_shape(1, T, E, R, H), I, x, idx, w, *w13, *w2, hq, hs, out,
                            status, stream=stream)
            for r, a, off, q, s in zip(rows, coded, offs, qs, ss):
                m.moe_expert_gemm_swiglu(m.make_shape(1, r, E, 1, H, r), I, H, *a, off, *w13, q, s,
                                         stream=stream)
            m.moe_rmsnorm(m.make_shape(1, T, 1, 1, H), x, x[0], 1e-6, y=y, stream=stream)
        stream.synchronize()
        return [out, y, *qs, *ss]
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
