"""moe_expert_gemm and moe_expert_gemm_swiglu by each of their ways (few rows; tiles
of 128 rows; tiles that two CTAs share): every test says which way its sizes have
to go and asks the rule, so that another rule cannot empty it."""
from __future__ import annotations

import threading

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _ops as o
from ._plan import plan, sms, way
from .test_experts_gpu import check, layout, run_gemm, run_swiglu
from .test_operators_guard_gpu import Guarded

pytestmark = pytest.mark.gpu
BOTH = pytest.mark.parametrize("swiglu", [False, True])


def outputs(n, swiglu):
    """All outputs for `n` columns of y or of the activation."""
    return 2 * n if swiglu else n


def goes(want, N, cap, E, n, k, swiglu):
    p = plan(N, cap, E, n, k, swiglu, sms())
    assert way(p) == want, p
    return p


# ranks' group sizes, rows per rank, columns, k: one line for each way
WAYS = [
    ("few", [[9, 0, 30, 2]], 41, 256, 640),
    ("tiles", [[70, 0, 300, 41]], 411, 1280, 896),
    ("shared", [[130, 0, 300, 82]], 512, 1280, 4096),
]


def inputs(sizes, cap, n, k, swiglu, seed=0):
    N, E = len(sizes), len(sizes) * len(sizes[0])
    gen = torch.Generator().manual_seed(seed + n + k)
    return (m.make_shape(N, cap, E, 1, 128, cap), outputs(n, swiglu), o.make_rows(gen, N * cap, k),
            layout(sizes, cap), o.make_weights(gen, E, outputs(n, swiglu), k))


@BOTH
@pytest.mark.parametrize("want,sizes,cap,n,k", WAYS + [
    ("shared", [[3, 0, 70], [0, 131, 1]], 140, 1024, 4096),
    ("shared", [[300]], 300, 1408, 4224),      # halves of 16 and 17 k blocks
    ("shared", [[129]], 200, 1664, 8192),
    ("tiles", [[33, 0, 31, 32], [64, 200, 0, 1]], 300, 1408, 640),
])
def test_matches_formula(want, sizes, cap, n, k, swiglu):
    sh, n, a, off, w = inputs(sizes, cap, n, k, swiglu)
    goes(want, sh.N, cap, sh.E, n, k, swiglu)
    check(sh, n, k, a, off, w, swiglu)


@BOTH
@pytest.mark.parametrize("sizes,cap,n,k", [
    ([[2101]], 2101, 5760, 640),                           # 45 column blocks, 17 row tiles
    ([[5, 0, 2177, 640, 33]], 2900, 2944, 896),            # uneven groups, rows to spare
    ([[700, 1], [0, 900]], 1000, 3712, 384),
])
def test_tiles_follow_each_other_in_a_cta(sizes, cap, n, k, swiglu):
    """More tiles than SMs, so that rings, accumulators and scale buffers go on from
    one tile to the next, over k blocks that are no multiple of four; tiles of one
    column block among those of two; runs of row tiles and a short last one."""
    sh, n, a, off, w = inputs(sizes, cap, n, k, swiglu)
    p = goes("tiles", sh.N, cap, sh.E, n, k, swiglu)
    real = sum(-(-g // 128) for s in sizes for g in s) * -(-(n // 128) // 2)
    assert p.wide == 2 and real > sms() and (n // 128 % 2 == 1 or swiglu)
    check(sh, n, k, a, off, w, swiglu)


@BOTH
@pytest.mark.parametrize("want,sizes,cap,n,k", WAYS)
def test_nan_stays_in_its_row(want, sizes, cap, n, k, swiglu):
    """Rows of other groups, and past the received ones, may hold anything."""
    sizes = [[g - (i == 3) for i, g in enumerate(s)] for s in sizes]  # a row of no group
    sh, n, a, off, w = inputs(sizes, cap, n, k, swiglu)
    goes(want, sh.N, cap, sh.E, n, k, swiglu)
    run = run_swiglu if swiglu else run_gemm
    cols = n // 2 if swiglu else n
    clean = run(sh, cols, k, a, off, w)
    spoilt = [3, sizes[0][0] - 1, cap - 1]  # the last one is no group's
    for i, r in enumerate(spoilt):
        a[0][r] = 0x7F
        a[1][r] = (1.0, float("nan"), float("inf"))[i]
    dirty = run(sh, cols, k, a, off, w)
    keep = [i for i in range(cap) if i not in spoilt[:2]]
    if swiglu:
        assert torch.equal(clean[0][0, keep], dirty[0][0, keep])
        assert torch.equal(clean[1][0, keep], dirty[1][0, keep])
        for r in spoilt[:2]:
            assert dirty[1][0, r].isnan().all() and (dirty[0][0, r] & 0x7F == 0x7F).all()
    else:
        assert torch.equal(clean[0, keep].view(torch.int16), dirty[0, keep].view(torch.int16))
        assert dirty[0, spoilt[:2]].isnan().all()


@BOTH
@pytest.mark.parametrize("want,sizes,cap,n,k", WAYS)
def test_offsets_past_the_capacity_are_clipped(want, sizes, cap, n, k, swiglu):
    sh, n, a, off, w = inputs(sizes, cap, n, k, swiglu)
    goes(want, sh.N, cap, sh.E, n, k, swiglu)
    off[0, -1] += 1000
    off[0, -2] -= 7
    check(sh, n, k, a, off, w, swiglu)


@BOTH
@pytest.mark.parametrize("want,rows,n,k", [("shared", 512, 1280, 4096), ("tiles", 512, 1280, 640),
                                           ("few", 512, 128, 640)])
def test_offsets_that_name_rows_twice(want, rows, n, k, swiglu):
    """Two groups of all rows are more tiles than rows are, and on the ways with a
    group of CTAs to a unit more units than CTAs: the call ends inside its outputs,
    and the next one is right."""
    gen = torch.Generator().manual_seed(rows + n + k)
    cols, n = n, outputs(n, swiglu)
    p = goes(want, 1, rows, 4, n, k, swiglu)
    at = 16 if want == "few" else 128
    assert 2 * (rows // at) > p.units
    a = [t.cuda() for t in o.make_rows(gen, rows, k)]
    w = [t.cuda() for t in o.make_weights(gen, 4, n, k)]
    sh, g = m.make_shape(1, rows, 4, 1, 128, rows), Guarded()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = ([g((rows, cols), torch.uint8), g((rows, cols // 128), torch.float32)] if swiglu
            else [g((rows, cols), torch.bfloat16)])

    def call(off):
        off = torch.tensor([off], dtype=torch.int32).cuda()
        (m.moe_expert_gemm_swiglu if swiglu else m.moe_expert_gemm)(sh, cols, k, *a, off, *w, *outs,
                                                                     status)
    call([0, rows, 0, rows, 0])
    g.check()
    assert int(status) == 0
    call([0, rows, rows, rows, rows])
    torch.cuda.synchronize()
    p, err = o.product64(a[0].cpu(), a[1].cpu(), w[0][0].cpu(), w[1][0].cpu())
    if swiglu:
        o.assert_codes(*[t.cpu() for t in outs], *o.swiglu64(p, err))
    else:
        o.assert_bf16(outs[0], p, err)


@BOTH
@pytest.mark.parametrize("edge", ["32 rows", "a CTA an SM", "8 rows an expert"])
def test_both_sides_of_the_rules_edges(edge, swiglu):
    """The smallest step over each bound of the rule changes the way, and both ways
    give the formula's rows."""
    half = 2 if swiglu else 1
    if edge == "32 rows":
        E, k, nb = 1, 256, -(-sms() // 3)
        sides = [(32, nb), (33, nb)]  # 33 rows are three groups of 16
    elif edge == "a CTA an SM":
        E, k = 1, 384
        nb = -(-sms() // 4) - 1       # 64 rows are four
        sides = [(64, nb), (64, nb + 1)]
    else:
        E, k = 8, 4096 // half
        sides = [(64, 24), (65, 24)]
    nb_even = [(rows, nb + (nb % 2 if swiglu else 0)) for rows, nb in sides]
    if edge == "a CTA an SM" and swiglu:
        nb_even = [(64, sides[0][1] // 2 * 2), (64, sides[0][1] // 2 * 2 + 2)]
    for (rows, nb), few in zip(nb_even, (True, False)):
        n = 128 * nb
        assert plan(1, rows, E, n, k, swiglu, sms()).few == few, (rows, nb)
        gen = torch.Generator().manual_seed(rows + nb)
        sizes = [[rows]] if E == 1 else [[7, 9, 0, 20, 8, 1, 10, rows - 55]]
        check(m.make_shape(1, rows, E, 1, 128, rows), n, k, o.make_rows(gen, rows, k),
              layout(sizes, rows), o.make_weights(gen, E, n, k), swiglu)


def caller(want, sizes, cap, n, k, swiglu):
    """(call(stream), outputs) of one product on the device."""
    sh, n, a, off, w = inputs(sizes, cap, n, k, swiglu)
    goes(want, sh.N, cap, sh.E, n, k, swiglu)
    a, w, off = [t.cuda() for t in a], [t.cuda() for t in w], off.cuda()
    cols = n // 2 if swiglu else n
    outs = ([torch.zeros((cap, cols), dtype=torch.uint8, device="cuda"),
             torch.zeros((cap, cols // 128), device="cuda")] if swiglu
            else [torch.zeros((cap, cols), dtype=torch.bfloat16, device="cuda")])
    f = m.moe_expert_gemm_swiglu if swiglu else m.moe_expert_gemm

    def call(stream=None, into=outs):
        f(sh, cols, k, *a, off, *w, *into, stream=stream)
    return call, outs


@BOTH
@pytest.mark.parametrize("want,sizes,cap,n,k", WAYS)
def test_repeats_streams_and_graphs_are_identical(want, sizes, cap, n, k, swiglu):
    call, outs = caller(want, sizes, cap, n, k, swiglu)
    call()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        call(st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, first))
    for t in outs:
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, first))


@BOTH
def test_all_ways_at_once_from_host_threads(swiglu):
    """A thread and a stream for each way, twice over."""
    made = [caller(*w, swiglu) for w in WAYS]
    want = []
    for call, outs in made:
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    got, errors = {}, []

    def work(i):
        try:
            torch.cuda.set_device(0)
            call, outs = made[i % len(made)]
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                mine = [torch.zeros_like(t) for t in outs]
            for _ in range(20):
                call(st, mine)
            st.synchronize()
            got[i] = mine
        except Exception as e:  # reported by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2 * len(made))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(2 * len(made)):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i % len(made)]))


@pytest.mark.parametrize("rows,H,inter,ways", [
    (24, 256, 256, ("few", "few")),
    (300, 1280, 1408, ("tiles", "tiles")),
    (300, 4096, 1280, ("shared", "tiles")),
    (200, 2048, 4096, ("tiles", "shared")),
])
def test_calls_follow_each_other_on_a_stream(rows, H, inter, ways):
    """Programmatic launches: each call's inputs are those that the call before it
    made, over and over without a wait on the host, directly and as a graph."""
    gen = torch.Generator().manual_seed(rows + H)
    goes(ways[0], 1, rows, 1, 2 * inter, H, True)
    goes(ways[1], 1, rows, 1, H, inter, False)
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    w13 = [t.cuda() for t in o.make_weights(gen, 1, 2 * inter, H)]
    w2 = [t.cuda() for t in o.make_weights(gen, 1, H, inter)]
    x0 = o.bf16(torch.randn((rows, H), generator=gen)).cuda()
    sh = m.make_shape(1, rows, 1, 1, H, rows)
    x = torch.empty_like(x0)
    q = torch.empty((rows, H), dtype=torch.uint8, device="cuda")
    s = torch.empty((rows, H // 128), device="cuda")
    hq = torch.empty((rows, inter), dtype=torch.uint8, device="cuda")
    hs = torch.empty((rows, inter // 128), device="cuda")
    y = torch.empty_like(x0)

    def chain(sync):
        x.copy_(x0)
        for _ in range(15):
            m.moe_rmsnorm(sh, x, gamma, 1e-6, q=q, s=s)
            sync()
            m.moe_expert_gemm_swiglu(sh, inter, H, q, s, None, *w13, hq, hs)
            sync()
            m.moe_expert_gemm(sh, H, inter, hq, hs, None, *w2, y)
            sync()
            m.moe_rmsnorm(sh, y, gamma, 1e-6, res=x, res_out=x)
            sync()
        return x.clone()
    want = chain(torch.cuda.synchronize)
    assert want.isfinite().all() and not torch.equal(want, x0)
    assert torch.equal(chain(lambda: None), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain(lambda: None)
    x.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want)
