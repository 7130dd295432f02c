"""The norm, the dispatch, the experts, the combine and the few-token layer as one
path: against each other and against 64 bits."""
from __future__ import annotations

import os
import sys

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _ops as o

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def layer64(x, idx, w, w13, w2, hq, hs, row_of):
    """The path's output from its own coded activations, and its error's bound:
    each expert's output is rounded to bf16, then weighted and added in fp32."""
    H, I = x.shape[-1], w2[0].shape[-1]
    want = torch.zeros(x.shape, dtype=torch.float64)
    err = torch.zeros_like(want)
    for t in range(idx.shape[0]):
        for k in range(idx.shape[1]):
            e, row = int(idx[t, k]), row_of(t, k)
            p, pe = o.product64(hq[row][None], hs[row][None], w2[0][e], w2[1][e])
            y = p[0].abs()
            want[t] += float(w[t, k]) * p[0]
            err[t] += float(w[t, k]) * (pe[0] + (y + pe[0]) * 2.0 ** -8 + 2 * idx.shape[1] * o.U * y)
    return want, err


@pytest.mark.parametrize("N,T,E,R,H,I", [(2, 9, 8, 3, 256, 128), (4, 33, 16, 4, 512, 256)])
def test_experts_between_dispatch_and_combine(N, T, E, R, H, I):
    gen = torch.Generator().manual_seed(N * T)
    x = o.bf16(torch.randn((N, T, H), generator=gen))
    idx = torch.rand((N, T, E), generator=gen).topk(R, dim=-1).indices.int()
    w = torch.rand((N, T, R), generator=gen)
    w = w / w.sum(-1, keepdim=True)
    w13, w2 = o.make_weights(gen, E, 2 * I, H), o.make_weights(gen, E, H, I)
    buf = m.MoeBuffers(N, T, E, R, H)
    dw13, dw2 = [t.cuda() for t in w13], [t.cuda() for t in w2]
    xd, idxd, wd = x.cuda(), idx.cuda(), w.cuda()
    buf.dispatch(xd, idxd)
    buf.experts(*dw13, *dw2)
    buf.combine(idxd, wd)
    torch.cuda.synchronize()
    assert int(buf.status) == 0
    # every grouped row's activations
    off, src = buf.grp_off.cpu(), buf.grp_src.cpu()
    xq, xs = o.code_rows(x.view(N * T, H))
    Er, at = E // N, {}
    for r in range(N):
        for j in range(Er):
            for i in range(int(off[r, j]), int(off[r, j + 1])):
                at[(int(src[r, i, 0]) * T + int(src[r, i, 1]), r * Er + j)] = (r, i)
    hq, hs = buf.h_q.cpu(), buf.h_s.cpu()
    for (t, e), (r, i) in at.items():
        p, pe = o.product64(xq[t][None], xs[t][None], w13[0][e], w13[1][e])
        h, he = o.swiglu64(p, pe)
        o.assert_codes(hq[r, i][None], hs[r, i][None], h, he)
    flat = idx.view(N * T, R)
    want, err = layer64(x.view(N * T, H), flat, w.view(N * T, R), w13, w2, hq, hs,
                        lambda t, k: at[(t, int(flat[t, k]))])
    o.assert_bf16(buf.out.view(N * T, H), want, err)


def test_example_agrees_with_itself():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_layer
    # each path is within 2^-8 of the same sums (bf16 of the expert outputs, of the
    # sum), but the codes of h may differ by a step where a value is near a tie
    assert moe_layer.main(["--ranks", "4", "--tokens", "40", "--hidden", "1024", "--experts", "16",
                           "--topk", "4", "--inter", "384"]) < 2 ** -7


def test_rows_around_the_narrow_kernel_agree():
    """Sixteen rows in all go one way, seventeen another: the same rows come out
    within the products' error."""
    gen = torch.Generator().manual_seed(11)
    k, n = 640, 512
    a, w = o.make_rows(gen, 17, k), o.make_weights(gen, 1, n, k)
    d = [t.cuda() for t in (*a, *w)]
    ys = []
    for rows in (16, 17):
        y = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
        m.moe_expert_gemm(m.make_shape(1, rows, 1, 1, 128, rows), n, k, d[0], d[1], None, d[2],
                          d[3], y)
        ys.append(y.cpu())
    p, err = o.product64(a[0], a[1], w[0][0], w[1][0])
    o.assert_bf16(ys[0], p[:16], err[:16])
    o.assert_bf16(ys[1], p, err)


@pytest.mark.parametrize("rows", [7, 700])
def test_many_experts(rows):
    """1024 experts, most of them empty."""
    gen = torch.Generator().manual_seed(rows)
    E, n, k = 1024, 128, 128
    sizes = torch.bincount(torch.randint(0, E, (rows,), generator=gen), minlength=E)
    off = torch.zeros((1, E + 1), dtype=torch.int32)
    off[0, 1:] = sizes.cumsum(0)
    a, w = o.make_rows(gen, rows, k), o.make_weights(gen, E, n, k)
    y = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
    m.moe_expert_gemm(m.make_shape(1, rows, E, 1, 128, rows), n, k, a[0].cuda(), a[1].cuda(),
                      off.cuda(), w[0].cuda(), w[1].cuda(), y)
    e = torch.repeat_interleave(torch.arange(E), sizes)
    av, wv = o.rows64(*a), o.weights64(*w)[e]
    p = (wv @ av[:, :, None])[..., 0]
    err = o.gamma(1) * (wv.abs() @ av.abs()[:, :, None])[..., 0]
    o.assert_bf16(y, p, err)


def test_calls_follow_each_other_on_a_stream():
    """Programmatic launches: each call's inputs are the call's before it, over and
    over without a wait on the host."""
    gen = torch.Generator().manual_seed(12)
    rows, k = 24, 256
    gamma = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    w13 = [t.cuda() for t in o.make_weights(gen, 1, 2 * k, k)]
    w2 = [t.cuda() for t in o.make_weights(gen, 1, k, k)]
    x0 = o.bf16(torch.randn((rows, k), generator=gen)).cuda()
    sh = m.make_shape(1, rows, 1, 1, k, rows)

    def chain(sync):
        x = x0.clone()
        q = torch.empty((rows, k), dtype=torch.uint8, device="cuda")
        s = torch.empty((rows, k // 128), device="cuda")
        hq, hs = torch.empty_like(q), torch.empty_like(s)
        y = torch.empty_like(x)
        for _ in range(30):
            m.moe_rmsnorm(sh, x, gamma, 1e-6, q=q, s=s)
            sync()
            m.moe_expert_gemm_swiglu(sh, k, k, q, s, None, *w13, hq, hs)
            sync()
            m.moe_expert_gemm(sh, k, k, hq, hs, None, *w2, y)
            sync()
            m.moe_rmsnorm(sh, y, gamma, 1e-6, res=x, res_out=x)
            sync()
        return x
    assert torch.equal(chain(lambda: None), chain(torch.cuda.synchronize))


def test_a_graph_keeps_its_activations_when_another_width_is_called():
    """A captured layer is replayed after calls with other experts on the same
    buffers and with new tensors in memory."""
    gen = torch.Generator().manual_seed(13)
    N, T, E, R, H = 2, 24, 8, 2, 512
    x = o.bf16(torch.randn((N, T, H), generator=gen)).cuda()
    idx = torch.rand((N, T, E), generator=gen).topk(R, dim=-1).indices.int().cuda()
    w = torch.rand((N, T, R), generator=gen).cuda()
    wide, narrow = ([t.cuda() for t in (*o.make_weights(gen, E, 2 * I, H),
                                        *o.make_weights(gen, E, H, I))] for I in (512, 128))
    buf = m.MoeBuffers(N, T, E, R, H)

    def layer(weights, stream=None):
        buf.dispatch(x, idx, stream=stream)
        buf.experts(*weights, stream=stream)
        return buf.combine(idx, w, stream=stream)
    want = layer(wide).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(wide)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = layer(narrow, side)
    torch.cuda.current_stream().wait_stream(side)
    other = other.clone()
    rows = N * buf.cap
    # the sizes of the first width's buffers: what the allocator would give again
    new = [torch.full((rows * 512,), 0x5C, dtype=torch.uint8, device="cuda") for _ in range(4)]
    new += [torch.full((rows * 16,), 0x5C, dtype=torch.uint8, device="cuda") for _ in range(4)]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(buf.out, want) and not torch.equal(other, want)
    assert all((t == 0x5C).all() for t in new)
    side.wait_stream(torch.cuda.current_stream())
    again = layer(narrow, side)
    side.synchronize()
    assert torch.equal(again, other)
