"""64-bit forms of the norm, the experts' products and the few-token layer, with
bounds on how far 32-bit arithmetic may be from them (CPU, torch float64).

Bounds, with u = 2^-24 the relative error of one fp32 operation:
  * a product's block of 128: e4m3 products are exact, their sum goes through
    at most 128 fp32 additions, each of which may truncate (2 u of the sum of
    magnitudes): 128 * 2 u = 2^-16 of it; the scaling and the Kb block sums add
    2 u + Kb u.  GAMMA(Kb) = 2^-16 + (Kb + 2) * 2^-24, times the sum of
    magnitudes;
  * silu(g) * u: |d silu/dg| <= 1.1, so 1.1 |u| dg + |silu(g)| du, plus six
    fp32 operations and the 2-ulp exponential: 16 u |h|;
  * a bf16 result: half a step, at most 2^-8 of the value for values at the low
    end of a binade (2^-9 of the binade's top), plus the smallest subnormal;
  * a code: the nearest e4m3 value, where v / s may be off by the error of v.
"""
from __future__ import annotations

import numpy as np
import torch

BLOCK = 128
U = 2.0 ** -24


def gamma(kb: int) -> float:
    return 2.0 ** -16 + (kb + 2) * U


def bf16(a) -> torch.Tensor:
    return torch.as_tensor(a).to(torch.bfloat16)


def values(q: torch.Tensor) -> torch.Tensor:
    return q.cpu().view(torch.float8_e4m3fn).double()


def rows64(q, s) -> torch.Tensor:
    return values(q) * s.cpu().double().repeat_interleave(BLOCK, -1)


def weights64(q, s) -> torch.Tensor:
    s = s.cpu().double()
    return values(q) * s.repeat_interleave(BLOCK, -1).repeat_interleave(BLOCK, -2)


def code_rows(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """The dispatch's coding of bf16 rows with IEEE fp32 divisions: bytes, scales."""
    v = x.cpu().float().numpy()
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    s = np.abs(b).max(-1) / np.float32(448.0)
    safe = np.where(s > 0, s, np.float32(1.0))[..., None]
    q = torch.from_numpy(np.where(s[..., None] > 0, b / safe, np.float32(0.0)).reshape(v.shape))
    return q.to(torch.float8_e4m3fn).view(torch.uint8), torch.from_numpy(s)


def make_rows(gen, rows: int, k: int) -> tuple[torch.Tensor, torch.Tensor]:
    return code_rows(bf16(torch.randn((rows, k), generator=gen)))


def make_weights(gen, E: int, n: int, k: int) -> tuple[torch.Tensor, torch.Tensor]:
    q = (torch.randn((E, n, k), generator=gen) * 110).clamp(-448, 448)
    s = 0.75 + 0.5 * torch.rand((E, n // BLOCK, k // BLOCK), generator=gen)
    return q.to(torch.float8_e4m3fn).view(torch.uint8), s / (110 * k ** 0.5)


def assert_bf16(got: torch.Tensor, want: torch.Tensor, err) -> None:
    """got = bf16 of something within err of want."""
    g = got.cpu().double()
    bound = err + (want.abs() + err) * 2.0 ** -8 + 2.0 ** -133
    bad = ~((g - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), g[bad][:4], want[bad][:4])


def assert_codes(q: torch.Tensor, s: torch.Tensor, v: torch.Tensor, err) -> None:
    """(q, s) = the block-128 coding of something within err of v."""
    err = torch.as_tensor(err, dtype=torch.float64).expand(v.shape)
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    e = err.reshape(b.shape)
    s = s.cpu().double()
    amax = b.abs().amax(-1)
    assert ((s * 448 - amax).abs() <= e.amax(-1) + 4 * U * amax + 448 * 2.0 ** -149).all()
    z = s > 0
    assert (values(q).reshape(b.shape)[~z] == 0).all()
    t = (b / torch.where(z, s, 1.0)[..., None])[z]
    te = (e / torch.where(z, s, 1.0)[..., None])[z] + 4 * U * t.abs()
    got = values(q).reshape(b.shape)[z]
    _, exp = torch.frexp(got.abs().clamp(min=2.0 ** -6))
    step = torch.pow(2.0, (exp - 4).double())  # of got's binade: the wider side
    far = (got - t).abs() - te
    assert (far <= step / 2 * (1 + 1e-9)).all(), far.max()


def product64(a_q, a_s, w_q, w_s) -> tuple[torch.Tensor, torch.Tensor]:
    """Rows times weights^T, and the bound on the fp32 result's error."""
    a, w = rows64(a_q, a_s), weights64(w_q, w_s)
    return a @ w.T, gamma(a.shape[-1] // BLOCK) * (a.abs() @ w.abs().T)


def swiglu64(p: torch.Tensor, err: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    g, u = p.chunk(2, -1)
    dg, du = err.chunk(2, -1)
    silu = g * torch.sigmoid(g)
    h = silu * u
    return h, 1.1 * u.abs() * dg + silu.abs() * du + 1.1 * dg * du + 16 * U * h.abs()
