"""moe_expert_gemm and moe_expert_gemm_swiglu on the GPU against the products
in 64 bits, group by group."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _ops as o

pytestmark = pytest.mark.gpu
SENT = 0x7FA5


def layout(sizes_by_rank, cap):
    off = torch.zeros((len(sizes_by_rank), len(sizes_by_rank[0]) + 1), dtype=torch.int32)
    for r, sizes in enumerate(sizes_by_rank):
        off[r, 1:] = torch.tensor(sizes).cumsum(0)
    return off


def run_gemm(sh, n, k, a, off, w):
    y = torch.empty((sh.N, sh.cap, n), dtype=torch.bfloat16, device="cuda")
    y.view(torch.int16).fill_(SENT)
    m.moe_expert_gemm(sh, n, k, a[0].cuda(), a[1].cuda(), None if off is None else off.cuda(),
                      w[0].cuda(), w[1].cuda(), y)
    torch.cuda.synchronize()
    return y.cpu()


def run_swiglu(sh, inter, k, a, off, w):
    hq = torch.full((sh.N, sh.cap, inter), 0xA5, dtype=torch.uint8, device="cuda")
    hs = torch.full((sh.N, sh.cap, inter // 128), -1.0, device="cuda")
    m.moe_expert_gemm_swiglu(sh, inter, k, a[0].cuda(), a[1].cuda(),
                             None if off is None else off.cuda(), w[0].cuda(), w[1].cuda(), hq,
                             hs)
    torch.cuda.synchronize()
    return hq.cpu(), hs.cpu()


def groups(sh, off):
    """(rank, rows, expert) of every expert, clipped to cap."""
    Er = sh.E // sh.N
    for r in range(sh.N):
        for j in range(Er):
            b, t = (0, sh.cap) if off is None else (int(off[r, j]), int(off[r, j + 1]))
            b = min(max(b, 0), sh.cap)
            yield r, slice(b, min(max(t, b), sh.cap)), r * Er + j


def check(sh, n, k, a, off, w, swiglu):
    aq, as_ = a[0].view(sh.N, sh.cap, k), a[1].view(sh.N, sh.cap, k // 128)
    seen = torch.zeros((sh.N, sh.cap), dtype=torch.bool)
    if swiglu:
        hq, hs = run_swiglu(sh, n // 2, k, a, off, w)
    else:
        y = run_gemm(sh, n, k, a, off, w)
    for r, at, e in groups(sh, off):
        seen[r, at] = True
        if at.stop == at.start:
            continue
        p, err = o.product64(aq[r, at], as_[r, at], w[0][e], w[1][e])
        if swiglu:
            h, he = o.swiglu64(p, err)
            o.assert_codes(hq[r, at], hs[r, at], h, he)
        else:
            o.assert_bf16(y[r, at], p, err)
    if swiglu:
        assert (hq[~seen] == 0xA5).all() and (hs[~seen] == -1).all()
    else:
        assert (y.view(torch.int16)[~seen] == SENT).all()


CASES = [  # sizes of every rank's experts, rows per rank (0: the sum), n, k
    ([[1]], 0, 128, 128),
    ([[1]], 0, 256, 7168),
    ([[129]], 0, 384, 256),
    ([[127, 1, 0, 2]], 0, 256, 384),
    ([[0, 0, 0, 5]], 0, 512, 128),
    ([[0, 0, 0, 0]], 9, 256, 256),
    ([[33, 0, 31, 32], [64, 200, 0, 1]], 300, 768, 640),
    ([[128, 256, 64, 65]], 0, 1024, 512),
    ([[1] * 64], 0, 256, 1024),
    ([[300, 17, 260, 100]], 0, 1280, 896),
]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("sizes,cap,n,k", CASES)
def test_matches_formula(sizes, cap, n, k, swiglu):
    if swiglu and n % 256:
        n += 128
    N, Er = len(sizes), len(sizes[0])
    cap = cap or max(sum(s) for s in sizes)
    gen = torch.Generator().manual_seed(N * 7 + Er * 31 + n + k)
    sh = m.make_shape(N, cap, N * Er, 1, 128, cap)
    check(sh, n, k, o.make_rows(gen, N * cap, k), layout(sizes, cap),
          o.make_weights(gen, N * Er, n, k), swiglu)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,n,k", [(1, 512, 256), (77, 256, 1152), (513, 768, 384)])
def test_dense(M, n, k, swiglu):
    gen = torch.Generator().manual_seed(M + n + k)
    check(m.make_shape(1, M, 1, 1, 128, M), n, k, o.make_rows(gen, M, k), None,
          o.make_weights(gen, 1, n, k), swiglu)


@pytest.mark.parametrize("swiglu", [False, True])
def test_one_expert_a_rank_without_offsets(swiglu):
    gen = torch.Generator().manual_seed(3)
    check(m.make_shape(3, 41, 3, 1, 128, 41), 256, 256, o.make_rows(gen, 3 * 41, 256), None,
          o.make_weights(gen, 3, 256, 256), swiglu)


@pytest.mark.parametrize("swiglu", [False, True])
def test_offsets_past_the_capacity_are_clipped(swiglu):
    gen = torch.Generator().manual_seed(4)
    off = torch.tensor([[0, 20, 70, 90, 400]], dtype=torch.int32)
    check(m.make_shape(1, 64, 4, 1, 128, 64), 256, 256, o.make_rows(gen, 64, 256), off,
          o.make_weights(gen, 4, 256, 256), swiglu)


@pytest.mark.parametrize("swiglu", [False, True])
def test_nan_stays_in_its_row(swiglu):
    """Rows of other groups and past the received ones may hold anything."""
    gen = torch.Generator().manual_seed(5)
    sizes, cap, n, k = [[5, 40]], 60, 256, 256
    sh, off = m.make_shape(1, cap, 2, 1, 128, cap), layout(sizes, cap)
    a, w = o.make_rows(gen, cap, k), o.make_weights(gen, 2, n, k)
    run = run_swiglu if swiglu else run_gemm
    nn = n // 2 if swiglu else n
    clean = run(sh, nn, k, a, off, w)
    a[0][45:] = 0x7F
    a[1][45:] = float("inf")
    a[0][3] = 0x7F
    dirty = run(sh, nn, k, a, off, w)
    keep = [i for i in range(45) if i != 3]
    if swiglu:
        assert torch.equal(clean[0][0, keep], dirty[0][0, keep])
        assert torch.equal(clean[1][0, keep], dirty[1][0, keep])
        assert dirty[1][0, 3].isnan().all() and (dirty[0][0, 3] & 0x7F == 0x7F).all()
    else:
        assert torch.equal(clean[0, keep], dirty[0, keep])
        assert dirty[0, 3].isnan().all()


def test_extreme_gates():
    """Gates far below zero give zeros (not NaN), far above pass the up value."""
    k = 128
    a_q = torch.full((2, k), 0x38, dtype=torch.uint8)  # 1.0
    a_s = torch.ones((2, 1))
    a_s[1] = -1.0
    w_q = torch.full((1, 256, k), 0x38, dtype=torch.uint8)
    w_s = torch.tensor([[[0.5], [1.0 / 128]]])
    hq, hs = run_swiglu(m.make_shape(1, 2, 1, 1, 128, 2), 128, k, (a_q, a_s), None, (w_q, w_s))
    g = 64.0  # row 0: silu(64) * 1; row 1: silu(-64) * -1
    assert abs(float(hs[0, 0, 0]) * 448 - g) < 1e-4 and (hq[0, 0] == 0x7E).all()
    want = 64.0 * torch.exp(torch.tensor(-64.0, dtype=torch.float64))
    assert abs(float(hs[0, 1, 0]) * 448 / float(want) - 1) < 1e-4
    assert (hq[0, 1] == 0x7E).all()


def test_zero_rows_code_as_zeros():
    gen = torch.Generator().manual_seed(6)
    a = (torch.zeros((3, 256), dtype=torch.uint8), torch.zeros((3, 2)))
    w = o.make_weights(gen, 1, 512, 256)
    hq, hs = run_swiglu(m.make_shape(1, 3, 1, 1, 128, 3), 256, 256, a, None, w)
    assert hq.count_nonzero() == 0 and hs.count_nonzero() == 0


@pytest.mark.parametrize("swiglu", [False, True])
def test_repeats_streams_and_graphs_are_identical(swiglu):
    gen = torch.Generator().manual_seed(7)
    sizes, cap, n, k = [[70, 0, 130, 9]], 256, 512, 512
    sh, off = m.make_shape(1, cap, 4, 1, 128, cap), layout(sizes, cap).cuda()
    a, w = o.make_rows(gen, cap, k), o.make_weights(gen, 4, n, k)
    a, w = [t.cuda() for t in a], [t.cuda() for t in w]
    if swiglu:
        outs = [torch.zeros((cap, n // 2), dtype=torch.uint8, device="cuda"),
                torch.zeros((cap, n // 256), device="cuda")]

        def call(stream=None):
            m.moe_expert_gemm_swiglu(sh, n // 2, k, *a, off, *w, *outs, stream=stream)
    else:
        outs = [torch.zeros((cap, n), dtype=torch.bfloat16, device="cuda")]

        def call(stream=None):
            m.moe_expert_gemm(sh, n, k, *a, off, *w, *outs, stream=stream)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        call(st)
    st.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, want))
    for t in outs:
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, want))


def test_rows_past_32_bit_offsets():
    """A row buffer of more than 2^32 bytes: the last rows of the last rank."""
    N, cap, k, n = 2, 300_007, 8192, 128
    sh = m.make_shape(N, cap, N, 1, 128, cap)
    off = torch.tensor([[0, 0], [cap - 3, cap]], dtype=torch.int32)
    off[0] = torch.tensor([0, 2])
    gen = torch.Generator().manual_seed(8)
    q, s = o.make_rows(gen, 5, k)
    w = o.make_weights(gen, N, n, k)
    aq = torch.zeros((N, cap, k), dtype=torch.uint8, device="cuda")
    as_ = torch.zeros((N, cap, k // 128), device="cuda")
    aq[0, :2], as_[0, :2] = q[:2].cuda(), s[:2].cuda()
    aq[1, -3:], as_[1, -3:] = q[2:].cuda(), s[2:].cuda()
    y = torch.zeros((N, cap, n), dtype=torch.bfloat16, device="cuda")
    m.moe_expert_gemm(sh, n, k, aq, as_, off.cuda(), w[0].cuda(), w[1].cuda(), y)
    torch.cuda.synchronize()
    for rows, e, got in ((slice(0, 2), 0, y[0, :2]), (slice(2, 5), 1, y[1, -3:])):
        p, err = o.product64(q[rows], s[rows], w[0][e], w[1][e])
        o.assert_bf16(got, p, err)
    assert y[0, 2:].count_nonzero() == 0 and y[1, :-3].count_nonzero() == 0


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,n,k", [(20, 256, 4096), (129, 512, 4224), (300, 384, 4096),
                                   (40, 2304, 8192)])
def test_few_tiles_share_k(M, n, k, swiglu):
    """Few tiles and a long k: two CTAs have half of k each."""
    if swiglu and n % 256:
        n += 128
    gen = torch.Generator().manual_seed(M + n + k)
    check(m.make_shape(1, M, 1, 1, 128, M), n, k, o.make_rows(gen, M, k), None,
          o.make_weights(gen, 1, n, k), swiglu)


def test_few_tiles_share_k_in_groups():
    gen = torch.Generator().manual_seed(21)
    sizes, n, k = [[3, 0, 70], [0, 131, 1]], 512, 4096
    sh = m.make_shape(2, 140, 6, 1, 128, 140)
    check(sh, n, k, o.make_rows(gen, 280, k), layout(sizes, 140), o.make_weights(gen, 6, n, k),
          True)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,n,k", [(129, 2560, 4096), (300, 1024, 4224), (40, 7168, 4096),
                                   (33, 20480, 128)])
def test_wide_products_of_a_few_tiles(M, n, k, swiglu):
    gen = torch.Generator().manual_seed(M + n + k)
    check(m.make_shape(1, M, 1, 1, 128, M), n, k, o.make_rows(gen, M, k), None,
          o.make_weights(gen, 1, n, k), swiglu)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("sizes,cap,n,k", [
    ([[1000]], 0, 256, 512), ([[16, 17]], 0, 512, 1024), ([[40, 0, 17, 33]], 0, 256, 640),
    ([[5, 0], [31, 1], [0, 48]], 48, 256, 2048), ([[0, 0, 65, 0, 0, 1]], 66, 256, 128),
])
def test_more_rows_than_meet_the_weights_at_a_time(sizes, cap, n, k, swiglu):
    N, Er = len(sizes), len(sizes[0])
    cap = cap or max(sum(s) for s in sizes)
    gen = torch.Generator().manual_seed(N + Er + n + k)
    check(m.make_shape(N, cap, N * Er, 1, 128, cap), n, k, o.make_rows(gen, N * cap, k),
          layout(sizes, cap), o.make_weights(gen, N * Er, n, k), swiglu)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("sizes,cap,n,k", [
    ([[0, 1, 19, 0, 33, 2, 0, 5]], 64, 2560, 4096), ([[7, 0, 16, 1], [17, 12, 0, 0]], 30, 2560, 4096),
    ([[1, 0] * 150], 2000, 256, 2048),
])
def test_few_rows_an_expert(sizes, cap, n, k, swiglu):
    N, Er = len(sizes), len(sizes[0])
    gen = torch.Generator().manual_seed(N + Er + n + k)
    check(m.make_shape(N, cap, N * Er, 1, 128, cap), n, k, o.make_rows(gen, N * cap, k),
          layout(sizes, cap), o.make_weights(gen, N * Er, n, k), swiglu)
