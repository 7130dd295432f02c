"""What a kernel leaves whose bounded waits run out: MOE_ST_TIMEOUT, and no output
that those waits were for.  The library is compiled once more with the waits of
some CTAs giving up at once (the second of each cluster; where a launch has no
clusters, those of the second column block or tile), so nothing waits long and
nothing faults."""
from __future__ import annotations

import os

import pytest
import torch

from combine_expert_count_gb300 import build
from combine_expert_count_gb300 import moeroute as m

from . import _ops as o

pytestmark = pytest.mark.gpu
WHO = "(gridDim.z > 1 ? blockIdx.z == 1 : blockIdx.x == 1)"


@pytest.fixture(scope="module")
def path():
    return build.build(extra=[f"-DMOE_GIVE_UP={WHO}"],
                       out=os.path.join(build.BUILD, "libmoeroute_give_up.so"))


@pytest.fixture
def giving_up(path, monkeypatch):
    m.lib()
    monkeypatch.setattr(m, "_LIB_PATH", path)
    monkeypatch.setattr(m, "_lib", None)
    m.lib()


def product(swiglu, rows, n, k, sizes=None, status=True):
    """(outputs, status, rows and weights) of one product over sentinels."""
    gen = torch.Generator().manual_seed(rows + n + k)
    E = len(sizes) if sizes else 1
    a = [t.cuda() for t in o.make_rows(gen, rows, k)]
    w = [t.cuda() for t in o.make_weights(gen, E, n, k)]
    off = torch.tensor([[0] + sizes], dtype=torch.int32).cumsum(1).int().cuda() if sizes else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sh = m.make_shape(1, rows, E, 1, 128, rows)
    if swiglu:
        outs = [torch.full((rows, n // 2), 0xA5, dtype=torch.uint8, device="cuda"),
                torch.full((rows, n // 256), -1.0, device="cuda")]
        m.moe_expert_gemm_swiglu(sh, n // 2, k, *a, off, *w, *outs, st if status else None)
    else:
        outs = [torch.full((rows, n), -7.0, dtype=torch.bfloat16, device="cuda")]
        m.moe_expert_gemm(sh, n, k, *a, off, *w, *outs, st if status else None)
    torch.cuda.synchronize()
    return [t.cpu() for t in outs], int(st), [t.cpu() for t in (*a, *w)]


def untouched(outs):
    return all((t == v).all() for t, v in zip(outs, [0xA5 if len(outs) == 2 else -7.0, -1.0]))


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("status", [True, False])
@pytest.mark.parametrize("rows,n,k,sizes", [
    (20, 256, 1024, None),                     # few rows, a cluster for each block
    (9, 512, 640, [4, 0, 5]),
    (512, 1280, 4096, [130, 0, 300, 82]),      # tiles that two CTAs share
    (300, 1536, 4224, None),
])
def test_no_part_of_a_cluster_stores(giving_up, rows, n, k, sizes, status, swiglu):
    outs, st, _ = product(swiglu, rows, n, k, sizes, status)
    assert untouched(outs)
    assert st == (m.MOE_ST_TIMEOUT if status else 0)


@pytest.mark.parametrize("rows,n,k,lost", [
    (20, 384, 128, (slice(0, 20), slice(128, 256))),      # few rows: the second column block
    (300, 2560, 256, (slice(128, 256), slice(0, 128))),   # tiles: the second row tile
])
def test_others_store_theirs(giving_up, rows, n, k, lost):
    (y,), st, (aq, as_, wq, ws) = product(False, rows, n, k)
    assert st == m.MOE_ST_TIMEOUT
    assert (y[lost] == -7.0).all()
    p, err = o.product64(aq, as_, wq[0], ws[0])
    kept = torch.ones_like(y, dtype=torch.bool)
    kept[lost] = False
    o.assert_bf16(y[kept], p[kept], err[kept])


def few(T, E, R, H, inter):
    gen = torch.Generator().manual_seed(T + H)
    x = o.bf16(torch.randn((T, H), generator=gen)).cuda()
    idx = torch.rand((T, E), generator=gen).topk(R, dim=-1).indices.int().cuda()
    w = torch.rand((T, R), generator=gen).cuda()
    w13 = [t.cuda() for t in o.make_weights(gen, E, 2 * inter, H)]
    w2 = [t.cuda() for t in o.make_weights(gen, E, H, inter)]
    hq = torch.full((T, R, inter), 0xA5, dtype=torch.uint8, device="cuda")
    hs = torch.full((T, R, inter // 128), 1.0, device="cuda")
    out = torch.full((T, H), -7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.moe_layer_few(m.make_shape(1, T, E, R, H), inter, x, idx, w, *w13, *w2, hq, hs, out, st)
    torch.cuda.synchronize()
    return hq.cpu(), out.cpu(), int(st), x


@pytest.mark.parametrize("T,E,R,H,inter", [
    (3, 8, 2, 512, 512),   # both kernels in clusters
    (1, 2, 1, 512, 256),   # the second kernel's CTAs are alone: most of them are told by the first
])
def test_a_layer_stores_no_output(giving_up, T, E, R, H, inter):
    hq, out, st, _ = few(T, E, R, H, inter)
    assert st == m.MOE_ST_TIMEOUT and (hq == 0xA5).all() and (out == -7.0).all()


def test_a_layer_of_more_tokens_stores_no_output(giving_up):
    """Where the output would be, x's coding stays."""
    hq, out, st, x = few(20, 8, 2, 512, 512)
    assert st == m.MOE_ST_TIMEOUT and (hq == 0xA5).all()
    raw = out.view(torch.uint8).view(20, 4, 256)
    assert torch.equal(raw[..., :128].reshape(20, 512), o.code_rows(x)[0])


@pytest.mark.parametrize("swiglu", [False, True])
def test_the_next_call_is_right(path, swiglu):
    """The library as it is, after one that gave up, on the same stream."""
    with pytest.MonkeyPatch.context() as mp:
        m.lib()
        mp.setattr(m, "_LIB_PATH", path)
        mp.setattr(m, "_lib", None)
        m.lib()
        assert product(swiglu, 20, 512, 1024)[1] == m.MOE_ST_TIMEOUT
        assert product(swiglu, 300, 1280, 4096)[1] == m.MOE_ST_TIMEOUT
    for rows, n, k in ((20, 512, 1024), (300, 1280, 4096)):
        outs, st, (aq, as_, wq, ws) = product(swiglu, rows, n, k)
        assert st == 0
        p, err = o.product64(aq, as_, wq[0], ws[0])
        if swiglu:
            o.assert_codes(*outs, *o.swiglu64(p, err))
        else:
            o.assert_bf16(outs[0], p, err)
