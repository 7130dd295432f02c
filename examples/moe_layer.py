"""One mixture-of-experts layer of a transformer, as a serving loop runs it.

    python examples/moe_layer.py [--ranks N] [--tokens T] [--hidden H]
                                 [--experts E] [--topk R] [--inter I]

The residual stream goes through moe_rmsnorm (addition and norm in one pass), a
router picks experts (moe_linear's fp32 logits, moe_topk), and the layer runs twice:

  * as a batch: moe_dispatch groups the coded rows by expert,
    moe_expert_gemm_swiglu and moe_expert_gemm are the experts, moe_combine
    brings the weighted sums back;
  * for its first tokens alone, as a decode step of a few sequences does:
    moe_layer_few, which reads nothing but the chosen experts' weights.

After the batch a shared expert with 16-bit weights (moe_linear_glu, and moe_linear
with the routed experts' output as its residual) and the block's end (moe_block_norm:
the norm after the layer, a gate of each channel, the residual and the next layer's
norm with its coding) complete the block.

The two use the same coded weights and the same roundings up to the batch's bf16
expert outputs, so their results agree; the difference is printed, and the time
of each as a CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from combine_expert_count_gb300 import moeroute as m  # noqa: E402


def coded_weights(E: int, n: int, k: int, gen) -> tuple[torch.Tensor, torch.Tensor]:
    """Random weights [E][n][k] as an 8-bit checkpoint holds them: e4m3 and one
    scale for each block of 128 x 128."""
    w = torch.randn((E, n, k), generator=gen, device="cuda") / k ** 0.5
    b = w.view(E, n // 128, 128, k // 128, 128)
    s = b.abs().amax((2, 4)) / 448
    q = (b / s[:, :, None, :, None]).view(E, n, k).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), s


def graph_us(run, n: int = 20) -> float:
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        g.replay()
    start.record()
    for _ in range(n):
        g.replay()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) * 1e3 / n


def main(argv=None) -> float:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=64, help="tokens of each rank")
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=128)
    ap.add_argument("--topk", type=int, default=8)
    ap.add_argument("--inter", type=int, default=768)
    ap.add_argument("--shared", type=int, default=0, help="width of the shared expert (--inter's)")
    ap.add_argument("--few", type=int, default=8, help="tokens of the decode step")
    a = ap.parse_args(argv)
    N, T, H, E, R, I = a.ranks, a.tokens, a.hidden, a.experts, a.topk, a.inter
    gen = torch.Generator(device="cuda").manual_seed(0)

    def bf16(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    w13, w2 = coded_weights(E, 2 * I, H, gen), coded_weights(E, H, I, gen)
    router = bf16(E, H) / H ** 0.5
    gamma = 1 + bf16(H) / 8
    residual, attention = bf16(N, T, H), bf16(N, T, H)  # the stream, and what is added to it

    # the layer's input
    x = torch.empty_like(residual)
    m.moe_rmsnorm(m.make_shape(N, T, E, R, H), attention, gamma, 1e-6, y=x, res=residual,
                  res_out=residual)
    rows = m.make_shape(N, T, E, R, H)
    logits = torch.empty((N, T, E), device="cuda")
    idx = torch.empty((N, T, R), dtype=torch.int32, device="cuda")
    w = torch.empty((N, T, R), device="cuda")

    def route():
        m.moe_linear(rows, E, H, x, router, logits)
        m.moe_topk(rows, logits, idx, w)
    route()

    # the batch
    buf = m.MoeBuffers(N, T, E, R, H)

    def batch():
        buf.dispatch(x, idx)
        buf.experts(*w13, *w2)
        buf.combine(idx, w)
    batch_us = graph_us(batch)
    assert int(buf.status.item()) == 0

    # the rest of the block: the shared expert on top of the routed ones, and the end
    S = a.shared or I
    s13, s2 = bf16(2 * S, H) / H ** 0.5, bf16(H, S) / S ** 0.5
    post, gate, after = 1 + bf16(H) / 8, bf16(1, H) / 2, 1 + bf16(H) / 8
    h = torch.empty((N, T, S), dtype=torch.bfloat16, device="cuda")
    both, stream, nxt = (torch.empty_like(x) for _ in range(3))
    nxt_q = torch.empty((N, T, H), dtype=torch.uint8, device="cuda")
    nxt_s = torch.empty((N, T, H // 128), device="cuda")

    def block():
        route()
        batch()
        m.moe_linear_glu(rows, S, H, x, s13, h)
        m.moe_linear(rows, H, S, h, s2, both, res=buf.out, status=buf.status)
        m.moe_block_norm(rows, both, after, 1e-6, res_out=stream, y=nxt, q=nxt_q, s=nxt_s,
                         post_gamma=post, gate=gate, res=residual)
    block_us = graph_us(block)
    assert int(buf.status.item()) == 0 and bool(nxt.isfinite().all())

    # its first tokens alone
    few = min(a.few, T, m.MOE_FEW_MAX_TOKENS)
    xf, idxf, wf = x[0, :few].contiguous(), idx[0, :few].contiguous(), w[0, :few].contiguous()
    h_q = torch.empty((few, R, I), dtype=torch.uint8, device="cuda")
    h_s = torch.empty((few, R, I // 128), device="cuda")
    out, status = torch.empty_like(xf), torch.zeros(1, dtype=torch.int32, device="cuda")
    one = m.make_shape(1, few, E, R, H)

    def decode():
        m.moe_layer_few(one, I, xf, idxf, wf, *w13, *w2, h_q, h_s, out, status)
    few_us = graph_us(decode)
    assert int(status.item()) == 0

    off = float((out.float() - buf.out[0, :few].float()).norm() / out.float().norm())
    print(f"{N} ranks x {T} tokens, hidden {H}, {E} experts of {I}, top-{R}: "
          f"batch {batch_us:.1f} us (with router, shared expert and block end {block_us:.1f}), "
          f"{few} tokens alone {few_us:.1f} us, "
          f"their outputs differ by {off:.2g} of their norm")
    return off


if __name__ == "__main__":
    # the batch rounds each expert's output to bf16 (2^-9 each) before the sum
    sys.exit(0 if main() < 2 ** -7 else 1)
