"""The widest sizes that the calls around the experts take, and outputs onto both inputs."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from . import _dense as d
from . import _ops as o
from .test_block_norm_gpu import EPS, block, check, inputs

pytestmark = pytest.mark.gpu


def rand(gen, *shape, by=1.0):
    return (torch.randn(shape, generator=gen) * by).bfloat16().cuda()


@pytest.mark.parametrize("rows,n", [(1, 5), (3, 130), (40, 64), (300, 72)])
def test_longest_k(rows, n):
    k, gen = 65536, torch.Generator().manual_seed(rows)
    x, w, sh = rand(gen, rows, k), rand(gen, 2 * n, k, by=k ** -0.5), m.make_shape(1, rows, 1, 1, 128)
    one = w[:n].contiguous()
    for dtype in (torch.bfloat16, torch.float32):
        y = torch.empty((rows, n), dtype=dtype, device="cuda")
        m.moe_linear(sh, n, k, x, one, y)
        f32 = dtype == torch.float32
        (d.assert_f32 if f32 else o.assert_bf16)(y, *d.linear64(x, one, f32=f32))
    h = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
    m.moe_linear_glu(sh, n, k, x, w, h)
    o.assert_bf16(h, *d.glu64(x, w))


@pytest.mark.parametrize("rows", [1, 3])
def test_most_outputs(rows):
    n, k, gen = 1 << 20, 8, torch.Generator().manual_seed(rows)
    x, w, res = rand(gen, rows, k), rand(gen, n, k), rand(gen, rows, n)
    sh, y = m.make_shape(1, rows, 1, 1, 128), torch.empty_like(res)
    m.moe_linear(sh, n, k, x, w, y, res=res, act="relu")
    o.assert_bf16(y, *d.linear64(x, w, None, res, "relu"))
    h = torch.empty((rows, n // 2), dtype=torch.bfloat16, device="cuda")
    m.moe_linear_glu(sh, n // 2, k, x, w, h)
    o.assert_bf16(h, *d.glu64(x, w))


@pytest.mark.parametrize("rows,H", [(3, 2048), (400, 384), (330, 7168), (2, 65536)])
@pytest.mark.parametrize("swap", [False, True])
def test_both_outputs_onto_both_inputs(rows, H, swap):
    x, gamma, post, gate, res = inputs(rows, H)
    want = block(x, gamma, post=post, gate=gate, res=res)
    a, b = x.clone(), res.clone()
    got = block(a, gamma, post=post, gate=gate, res=b, res_out=a if swap else b, y=b if swap else a)
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_gate_of_each_row_of_a_long_batch():
    """As many rows of gate as rows, and a few: rows of several kernels' ways."""
    for rows, H, gates in ((3000, 256, 1500), (3000, 256, 3000), (1200, 4224, 300), (1200, 4224, 1200)):
        x, gamma, post, gate, res = inputs(rows, H, gates)
        kw = dict(post=post, gate=gate, res=res)
        check(block(x, gamma, eps=EPS, **kw), x, gamma, **kw)
