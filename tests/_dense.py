"""64-bit forms of the operators around the experts (16-bit products with their
epilogue, the router's choice, the block's end), with bounds on how far 32-bit
arithmetic may be from them.

Bounds, with u = 2^-24:
  * a product: bf16 products are exact, their sum goes through at most k fp32
    additions in the tensor cores, each of which may truncate (2 u of the sum of
    magnitudes), then at most 8 more of a cluster's parts and the bias: 2 (k + 8) u
    times the sum of magnitudes.  fp32 results: at most 512 such additions before a
    sum is taken out, then k / 512 that round: (1024 + k / 512 + 16) u;
  * an activation: its slope is at most 1.13, its value comes with (|v| + 16) 2 u; a
    gelu's exponential is of v^2 / 2, which adds v^2 2 u, and where the result is bf16
    its fitted polynomial is 2^-19 off; for v < 0 that is relative, above it less;
  * norms: the fp32 sum of H squares is at most H additions, the rest twelve
    operations; an error of v moves rstd by at most the mean of v's relative errors;
  * a bf16 result: half a step, at most 2^-8 of the value.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from ._ops import U


def act64(name: str, v: torch.Tensor) -> torch.Tensor:
    if name == "relu":
        return v.clamp(min=0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * torch.special.erfc(-v / math.sqrt(2)) / 2
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return torch.sigmoid(v) if name == "sigmoid" else v


def act_error(name: str, a: torch.Tensor, v: torch.Tensor, err: torch.Tensor,
              f32: bool = False) -> torch.Tensor:
    rel = (v.abs() + 16) * 2 * U
    if name == "gelu":
        rel = rel + v.square() * 2 * U + (0.0 if f32 else 2.0 ** -19)
    return 1.13 * err + rel * a.abs() + 2.0 ** -119


def product64(x, w, bias=None, f32=False):
    x, w = x.cpu().double(), w.cpu().double()
    p, mag, k = x @ w.T, x.abs() @ w.abs().T, x.shape[-1]
    if bias is not None:
        b = bias.cpu().double()
        p, mag = p + b, mag + b.abs()
    return p, ((1024 + k / 512 + 16) if f32 else 2 * (k + 8)) * U * mag


def linear64(x, w, bias=None, res=None, act="none", f32=False):
    """The formula, and the bound on the fp32 value's error before its last rounding."""
    p, err = product64(x, w, bias, f32)
    a = act64(act, p)
    err = act_error(act, a, p, err, f32) if act != "none" else err
    if res is not None:
        r = res.cpu().double()
        a, err = a + r, err + 2 * U * (a.abs() + r.abs())
    return a, err


def glu64(x, w13, bias=None, act="silu"):
    p, err = product64(x, w13, bias)
    (g, u), (dg, du) = p.chunk(2, -1), err.chunk(2, -1)
    a = act64(act, g)
    da = act_error(act, a, g, dg)
    return a * u, da * (u.abs() + du) + a.abs() * du + 2 * U * (a * u).abs()


def assert_f32(got: torch.Tensor, want: torch.Tensor, err) -> None:
    g = got.cpu().double()
    bound = err + U * (want.abs() + err) + 2.0 ** -149
    bad = ~((g - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), g[bad][:4], want[bad][:4])


def topk64(logits, R, bias=None, score="softmax", groups=1, kept=1, best=1, renorm=True,
           scale=1.0):
    """ids and weights (float64) of each row, by sorting whole rows in 64 bits."""
    l = logits.cpu().numpy().astype(np.float64)
    rows, E = l.shape
    per = E // groups
    with np.errstate(all="ignore"):
        top = l.max(-1, keepdims=True)
        if score == "softmax":
            s = np.where(l == -np.inf, 0.0, np.exp(l - top))
            s = s / s.sum(-1, keepdims=True)
        else:
            s = 1 / (1 + np.exp(-l))
        c = l if bias is None else s + bias.cpu().numpy().astype(np.float64)
        worth = s if bias is None and best == 2 else c
    out = (l == -np.inf) | np.isnan(c)
    c, worth = np.where(out, -np.inf, c), np.where(out, -np.inf, worth)
    idx, w = np.empty((rows, R), np.int64), np.empty((rows, R))
    for i in range(rows):
        g = np.sort(worth[i].reshape(groups, per), -1)[:, ::-1][:, :best].sum(-1)
        keep = np.argsort(-g, kind="stable")[:kept]
        e = np.sort(np.concatenate([np.arange(k * per, (k + 1) * per) for k in keep]))
        idx[i] = e[np.argsort(-c[i][e], kind="stable")[:R]]
        # out of service, by the logit or by the bias: no weight, and none taken
        lc = np.where(c[i, idx[i]] == -np.inf, -np.inf, l[i, idx[i]])
        chosen = np.where(lc == -np.inf, 0.0, s[i, idx[i]])
        if renorm and np.isfinite(lc.max()) and (score == "softmax" or lc.max() < 0):
            # the ratios of values that may be 0 by themselves
            chosen = np.exp(lc - lc.max()) / (1 + (np.exp(lc) if score == "sigmoid" else 0))
        total = chosen.sum()
        w[i] = scale * (chosen if not renorm else chosen / total if total > 0 else 0 * chosen)
    return torch.from_numpy(idx).int(), torch.from_numpy(w)


def topk_error(logits, w):
    """fp32's weights: exponentials of arguments that are |l - top| u off, sums of E."""
    l = logits.cpu().double()
    l = torch.where(l.isinf(), torch.zeros_like(l), l)
    reach = float(l.max() - l.min()) if l.numel() else 0.0
    return (reach + 64) * 2 * U * w.abs() + 2.0 ** -126


def block64(x, gamma, eps, post=None, gate=None, scale=1.0, res=None):
    """v, y and the bounds on their fp32 errors."""
    b = x.cpu().double()
    rows, H = b.shape
    err = torch.zeros_like(b)
    if post is not None:
        b = b * (b.square().mean(-1, keepdim=True) + eps).rsqrt() * post.cpu().double()
        err = (H / 2 + 12) * U * b.abs()
    if gate is not None:
        g = gate.cpu().double().repeat_interleave(rows // gate.shape[0], 0)
        b, err = b * g, err * g.abs() + U * (b * g).abs()
    v = b * scale + (res.cpu().double() if res is not None else 0.0)
    err = err * abs(scale) + U * v.abs()
    rstd = (v.square().mean(-1, keepdim=True) + eps).rsqrt()
    y = v * rstd * gamma.cpu().double()
    moved = err.square().mean(-1, keepdim=True).sqrt() * rstd  # of rstd, relatively
    yerr = err * rstd * gamma.cpu().double().abs() + ((H / 2 + 12) * U + moved) * y.abs()
    return v, err, y, yerr * 1.01
