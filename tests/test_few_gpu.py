"""moe_layer_few on the GPU: the coded activations that it leaves in its scratch
and the outputs, each against 64 bits."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _ops as o

pytestmark = pytest.mark.gpu


def inputs(T, E, R, H, inter, seed, idx=None):
    gen = torch.Generator().manual_seed(seed)
    x = o.bf16(torch.randn((T, H), generator=gen))
    if idx is None:
        idx = torch.rand((T, E), generator=gen).topk(R, dim=-1).indices.int()
    w = torch.rand((T, R), generator=gen)
    return x, idx, w / w.sum(-1, keepdim=True), o.make_weights(gen, E, 2 * inter, H), \
        o.make_weights(gen, E, H, inter)


def run(T, E, R, H, inter, x, idx, w, w13, w2, N=1):
    d = dict(device="cuda")
    hq = torch.full((T, R, inter), 0xA5, dtype=torch.uint8, **d)
    hs = torch.full((T, R, inter // 128), -1.0, **d)
    out = torch.full((T, H), 7.0, dtype=torch.bfloat16, **d)
    status = torch.full((1,), 99, dtype=torch.int32, **d)
    m.moe_layer_few(m.make_shape(N, T // N, E, R, H), inter, x.cuda(), idx.cuda(), w.cuda(),
                    w13[0].cuda(), w13[1].cuda(), w2[0].cuda(), w2[1].cuda(), hq, hs, out, status)
    torch.cuda.synchronize()
    return hq.cpu(), hs.cpu(), out.cpu(), int(status)


def check(T, E, R, H, inter, x, idx, w, w13, w2, N=1):
    hq, hs, out, status = run(T, E, R, H, inter, x, idx, w, w13, w2, N)
    xq, xs = o.code_rows(x)
    want = torch.zeros((T, H), dtype=torch.float64)
    err = torch.zeros((T, H), dtype=torch.float64)
    bad = False
    for t in range(T):
        first = {}
        for k in range(R):
            e = int(idx[t, k])
            if not 0 <= e < E:
                bad = True
                assert (hq[t, k] == 0xA5).all() and (hs[t, k] == -1).all()
                continue
            if e not in first:
                first[e] = k
                p, pe = o.product64(xq[t:t + 1], xs[t:t + 1], w13[0][e], w13[1][e])
                h, he = o.swiglu64(p, pe)
                o.assert_codes(hq[t, k:k + 1], hs[t, k:k + 1], h, he)
            s = first[e]
            p, pe = o.product64(hq[t, s:s + 1], hs[t, s:s + 1], w2[0][e], w2[1][e])
            wk = float(w[t, k])
            want[t] += wk * p[0]
            # the weighted sum adds R and the warps' eight partial sums
            err[t] += abs(wk) * (pe[0] + (R + 10) * o.U * pe[0] / o.gamma(inter // 128))
    o.assert_bf16(out, want, err)
    assert status == (m.MOE_ST_BAD_EXPERT if bad else 0)
    return out


@pytest.mark.parametrize("T,E,R,H,inter", [
    (1, 8, 2, 256, 128), (1, 1, 1, 128, 128), (1, 16, 8, 2048, 768), (2, 4, 4, 384, 256),
    (3, 60, 4, 1408, 256), (8, 8, 8, 256, 384), (9, 16, 3, 640, 128), (16, 5, 2, 256, 256),
    (17, 32, 8, 512, 256), (33, 12, 6, 256, 128), (64, 8, 2, 256, 128), (64, 64, 8, 384, 128),
])
def test_matches_formula(T, E, R, H, inter):
    check(T, E, R, H, inter, *inputs(T, E, R, H, inter, T * 1000 + E))


def test_every_token_on_one_expert():
    T, E, R, H, inter = 37, 6, 1, 256, 256
    idx = torch.full((T, R), 4, dtype=torch.int32)
    check(T, E, R, H, inter, *inputs(T, E, R, H, inter, 1, idx))


def test_bad_ids_are_skipped_and_flagged():
    T, E, R, H, inter = 5, 8, 3, 256, 128
    idx = torch.tensor([[0, 8, 1], [-1, -1, -1], [7, 6, 5], [2, 2 ** 31 - 1, 3], [4, 0, -5]],
                       dtype=torch.int32)
    out = check(T, E, R, H, inter, *inputs(T, E, R, H, inter, 2, idx))
    assert out[1].count_nonzero() == 0


def test_repeated_ids_of_a_token_add_their_weights():
    T, E, R, H, inter = 4, 5, 4, 256, 128
    idx = torch.tensor([[3, 3, 3, 3], [0, 1, 0, 1], [4, 3, 4, 2], [0, 0, 1, 2]],
                       dtype=torch.int32)
    check(T, E, R, H, inter, *inputs(T, E, R, H, inter, 3, idx))


def test_wide_rows():
    """Rows so wide that fewer than eight tokens are coded at a time."""
    T, E, R, H, inter = 5, 2, 1, 65536, 128
    check(T, E, R, H, inter, *inputs(T, E, R, H, inter, 4))


def test_ranks_are_only_a_view():
    a = inputs(12, 6, 2, 256, 128, 5)
    one = run(12, 6, 2, 256, 128, *a)
    three = run(12, 6, 2, 256, 128, *a, N=3)
    assert torch.equal(one[2], three[2]) and torch.equal(one[0], three[0])


def test_no_tokens_clears_the_status():
    x, idx, w, w13, w2 = inputs(1, 4, 2, 256, 128, 6)
    _, _, out, status = run(0, 4, 2, 256, 128, x[:0], idx[:0], w[:0], w13, w2)
    assert status == 0 and out.numel() == 0


def test_nan_stays_with_the_tokens_that_meet_it():
    T, E, R, H, inter = 6, 4, 2, 256, 128
    idx = torch.tensor([[0, 1], [1, 2], [2, 0], [0, 2], [3, 1], [1, 0]], dtype=torch.int32)
    x, idx, w, w13, w2 = inputs(T, E, R, H, inter, 7, idx)
    clean = run(T, E, R, H, inter, x, idx, w, w13, w2)[2]
    x2 = x.clone()
    x2[2, 5] = float("nan")
    w2_q = w2[0].clone()
    w2_q[3] = 0x7F  # an expert of token 4 alone
    dirty = run(T, E, R, H, inter, x2, idx, w, w13, (w2_q, w2[1]))[2]
    assert dirty[2].isnan().all() and dirty[4].isnan().all()
    keep = [0, 1, 3, 5]
    assert torch.equal(clean[keep], dirty[keep])


def test_repeats_streams_and_graphs_are_identical():
    T, E, R, H, inter = 11, 16, 4, 512, 256
    x, idx, w, w13, w2 = (t if isinstance(t, tuple) else t.cuda()
                          for t in inputs(T, E, R, H, inter, 8))
    w13, w2 = [t.cuda() for t in w13], [t.cuda() for t in w2]
    hq = torch.zeros((T, R, inter), dtype=torch.uint8, device="cuda")
    hs = torch.zeros((T, R, inter // 128), device="cuda")
    out = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sh = m.make_shape(1, T, E, R, H)

    def call(stream=None):
        m.moe_layer_few(sh, inter, x, idx, w, *w13, *w2, hq, hs, out, status, stream=stream)
    call()
    torch.cuda.synchronize()
    want = out.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        call(st)
    st.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [1, 4, 5, 17, 64])
def test_x_is_coded_as_the_dispatch_codes_it(T):
    """Gates of amax and up weights of one: h's codes are x's own, ties included."""
    gen = torch.Generator().manual_seed(T)
    amax = 448.0 / 2 ** torch.randint(0, 4, (T, 1), generator=gen).double()
    ties = (8.5 + torch.randint(0, 8, (T, 64), generator=gen)) * \
        2.0 ** torch.randint(-13, 5, (T, 64), generator=gen) * amax / 448
    any_ = amax * torch.rand((T, 63), generator=gen, dtype=torch.float64)
    x = torch.cat([amax, torch.cat([ties, any_], 1) *
                   (1 - 2 * torch.randint(0, 2, (T, 127), generator=gen))], 1)
    x[T // 2, 0] = 33.25  # no power of two between its scale and 1
    x[T // 2, 1:] = x[T // 2, 1:].clamp(-33.25, 33.25)
    x = o.bf16(x.float())
    w13 = torch.zeros((1, 256, 128), dtype=torch.uint8)
    w13[0, :128, 0] = 0x38  # 1.0
    w13[0, 128 + torch.arange(128), torch.arange(128)] = 0x38
    w2 = o.make_weights(gen, 1, 128, 128)
    hq, _, _, status = run(T, 1, 1, 128, 128, x, torch.zeros((T, 1), dtype=torch.int32),
                           torch.ones((T, 1)), (w13, torch.ones((1, 2, 1))), w2)
    want = o.code_rows(x)[0]
    assert status == 0 and torch.equal(hq[:, 0], torch.where(want == 0x80, 0, want))


@pytest.mark.parametrize("T", [3, 20])
def test_output_in_the_place_of_x(T):
    T, E, R, H, inter = T, 8, 3, 384, 256
    x, idx, w, w13, w2 = inputs(T, E, R, H, inter, 31)
    want = run(T, E, R, H, inter, x, idx, w, w13, w2)[2]
    d = [t.cuda() for t in (x, idx, w, *w13, *w2)]
    hq = torch.zeros((T, R, inter), dtype=torch.uint8, device="cuda")
    hs = torch.zeros((T, R, inter // 128), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.moe_layer_few(m.make_shape(1, T, E, R, H), inter, *d, hq, hs, d[0], status)
    torch.cuda.synchronize()
    assert torch.equal(d[0].cpu(), want)


@pytest.mark.parametrize("T", [2, 9])
def test_no_valid_id_gives_zeros(T):
    x, idx, w, w13, w2 = inputs(T, 4, 2, 256, 128, 32, torch.full((T, 2), 4, dtype=torch.int32))
    _, _, out, status = run(T, 4, 2, 256, 128, x, idx, w, w13, w2)
    assert status == m.MOE_ST_BAD_EXPERT and out.count_nonzero() == 0
