"""What the operators around the expert-parallel exchange are measured on.

Four operators of a mixture-of-experts layer: the norm that makes its input
(``norm``), the experts' two products over the rows that a dispatch groups
(``gemm``, and ``swiglu`` with the activation and the quantisation between the
products), and the whole layer for a few tokens (``few``).  Sizes are those of
this repository's configurations (hidden 7168 with 256 experts, hidden 2048
with 128 experts, top-8) with expert widths of 2048 and 768, and odd ones.

8-bit values are OCP e4m3; activations carry one fp32 scale per row and block
of 128 elements, weights one per block of 128 x 128.
"""
import collections
import math
import random

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
BLOCK = 128
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token's row between two layers while decoding
        dict(name="norm_one", op="norm", rows=1, H=7168, res=True, y=True, q=True),
        # a decode step of 16 ranks x 128 tokens, the bf16 row for the dispatch alone
        dict(name="norm_decode", op="norm", rows=2048, H=7168, res=True, y=True, q=False),
        # a prompt's tokens, bf16 for the dispatch and 8 bits for a shared expert; odd count
        dict(name="norm_prefill", op="norm", rows=32767, H=7168, res=True, y=True, q=True),
        # one token through a dense product (a shared expert's second one)
        dict(name="gemm_one", op="gemm", G=1, rows=1, n=7168, k=2048, skew=0.0),
        # second product of one rank's experts, decode batch: about 64 rows each
        dict(name="gemm_decode", op="gemm", G=32, rows=2048, n=7168, k=2048, skew=0.0),
        # a dense projection over a prompt of odd length
        dict(name="gemm_dense", op="gemm", G=1, rows=8191, n=7168, k=7168, skew=0.0),
        # first product, decode batch, hot and empty experts (hidden 2048)
        dict(name="swiglu_skew", op="swiglu", G=128, rows=1021, inter=768, k=2048, skew=1.0),
        # first product of one rank's experts, decode batch (hidden 7168)
        dict(name="swiglu_decode", op="swiglu", G=32, rows=2048, inter=2048, k=7168, skew=0.0),
        # first product of one rank's experts over a prompt, uneven experts
        dict(name="swiglu_prefill", op="swiglu", G=32, rows=32768, inter=2048, k=7168, skew=0.3),
        # the whole layer for one token (hidden 2048)
        dict(name="few_one", op="few", T=1, E=128, R=8, H=2048, inter=768),
        # the whole layer for a few tokens (hidden 7168, 256 experts)
        dict(name="few_four", op="few", T=4, E=256, R=8, H=7168, inter=2048),
        # the most tokens that still count as a few, every expert in use
        dict(name="few_many", op="few", T=32, E=64, R=8, H=7168, inter=2048),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _blocks(rng, lo, hi):
    """A multiple of 128 between lo and hi, spread over the logarithm."""
    v = BLOCK * _log(rng, lo // BLOCK, hi // BLOCK)
    return v + BLOCK if v in (1536, 3072) else v


def draw(rng):
    op = rng.choice(("norm", "gemm", "swiglu", "few"))
    if op == "norm":
        q = rng.random() < 0.7
        return dict(op=op, rows=_log(rng, 1, 32767), H=_blocks(rng, 128, 7168),
                    res=rng.random() < 0.7, y=not q or rng.random() < 0.7, q=q)
    if op == "few":
        E = rng.choice((8, 16, 60, 64, 128, 256))
        c = dict(op=op, T=_log(rng, 1, 32), E=E, R=rng.randint(1, 8), H=_blocks(rng, 256, 7168),
                 inter=_blocks(rng, 128, 2048))
        while E * c["H"] * c["inter"] > 64 * 7168 * 2048:  # no more weights than few_many's
            c["E"] = E = E // 2
        c["R"] = min(c["R"], E)
        return c
    G = _log(rng, 1, 128)
    c = dict(op=op, G=G, rows=_log(rng, 1, 32768), skew=rng.choice((0.0, 0.3, 1.0)))
    if op == "gemm":
        c.update(n=_blocks(rng, 128, 7168), k=_blocks(rng, 128, 7168))
        most, per = 8191 * 7168 * 7168, c["n"] * c["k"]
    else:
        c.update(inter=_blocks(rng, 128, 2048), k=_blocks(rng, 128, 7168))
        most, per = 32768 * 2048 * 7168, c["inter"] * c["k"]
    c["rows"] = max(1, min(c["rows"], most // per))
    while c["G"] * per * (1 if op == "gemm" else 2) > 32 * 4096 * 7168:
        c["G"] = max(1, c["G"] // 2)
    return c


def _group_sizes(case):
    """Rows of each group: shares of rank^-skew in a shuffled order, whole rows
    drawn by share (a fixed draw for each case: work() counts them too)."""
    G, rows = case["G"], case["rows"]
    r = random.Random(1000 * G + rows)
    share = [(i + 1) ** -case["skew"] for i in range(G)]
    r.shuffle(share)
    drawn = collections.Counter(r.choices(range(G), weights=share, k=rows))
    return [drawn[g] for g in range(G)]


# ------------------------------------------------------------------ inputs

def _dequant_rows(q, s):
    """[..., k] e4m3 bytes and [..., k/128] scales -> fp32."""
    v = q.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, BLOCK)) * s.unsqueeze(-1)).flatten(-2)


def _dequant_weights(q, s):
    """[..., n, k] e4m3 bytes and [..., n/128, k/128] scales -> fp32."""
    v = q.view(torch.float8_e4m3fn).float()
    v = v.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))
    return (v * s[..., :, None, :, None]).flatten(-2).flatten(-3, -2)


def _quant_rows(v):
    """fp32 [..., k] -> e4m3 bytes and scales amax/448 (0 for a zero block)."""
    b = v.unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1)
    s = amax / torch.full_like(amax, E4M3_MAX)  # by a tensor: a number becomes its reciprocal
    q = torch.where(s[..., None] > 0, b / s[..., None], torch.zeros_like(b))
    return q.to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2), s


def _weights(gen, E, n, k):
    """E experts' weights [E, n, k] as a checkpoint holds them: e4m3 values that
    fill the type's range and scales that bring them to a spread of 1/sqrt(k)."""
    w = torch.randn((E, n, k), generator=gen, device=DEVICE).mul_(110.0)
    q = w.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.rand((E, n // BLOCK, k // BLOCK), generator=gen, device=DEVICE)
    return q, (0.75 + 0.5 * s) / (110.0 * math.sqrt(k))


def _rows(gen, rows, k):
    """Activations with a few channels several times larger than the others."""
    x = torch.randn((rows, k), generator=gen, device=DEVICE)
    return x * (1 + 7 * (torch.rand(k, generator=gen, device=DEVICE) < 0.01))


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    st = dict(case=case)
    if case["op"] == "norm":
        rows, H = case["rows"], case["H"]
        st["x"] = _rows(gen, rows, H).bfloat16()
        st["res"] = (3 * _rows(gen, rows, H)).bfloat16() if case["res"] else None
        st["gamma"] = (1 + 0.2 * torch.randn(H, generator=gen, device=DEVICE)).bfloat16()
        st["res_out"] = torch.empty_like(st["x"]) if case["res"] else None
        st["y"] = torch.empty_like(st["x"]) if case["y"] else None
        st["q"] = torch.empty((rows, H), dtype=torch.uint8, device=DEVICE) if case["q"] else None
        st["s"] = torch.empty((rows, H // BLOCK), device=DEVICE) if case["q"] else None
        st["shape"] = (1, rows, 1, 1, H, 0)
        return st
    if case["op"] == "few":
        T, E, R, H, I = (case[c] for c in ("T", "E", "R", "H", "inter"))
        st["x"] = _rows(gen, T, H).bfloat16()
        p = torch.randn((T, E), generator=gen, device=DEVICE).softmax(-1)
        w, idx = p.topk(R, dim=-1)
        st["topk_w"] = w / w.sum(-1, keepdim=True)
        st["topk_idx"] = idx.int()
        st["w13_q"], st["w13_s"] = _weights(gen, E, 2 * I, H)
        st["w2_q"], st["w2_s"] = _weights(gen, E, H, I)
        st["h_q"] = torch.empty((T, R, I), dtype=torch.uint8, device=DEVICE)
        st["h_s"] = torch.empty((T, R, I // BLOCK), device=DEVICE)
        st["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEVICE)
        st["status"] = torch.zeros(1, dtype=torch.int32, device=DEVICE)
        st["shape"] = (1, T, E, R, H, 0)
        return st
    G, rows, k = case["G"], case["rows"], case["k"]
    sizes = _group_sizes(case)
    off = [0]
    for m in sizes:
        off.append(off[-1] + m)
    st["grp_off"] = torch.tensor([off], dtype=torch.int32, device=DEVICE)
    st["most"] = max(sizes)
    st["a_q"], st["a_s"] = _quant_rows(_rows(gen, rows, k))
    st["shape"] = (1, rows, G, 1, k, rows)
    if case["op"] == "gemm":
        st["w_q"], st["w_s"] = _weights(gen, G, case["n"], k)
        st["y"] = torch.empty((rows, case["n"]), dtype=torch.bfloat16, device=DEVICE)
    else:
        I = case["inter"]
        st["w_q"], st["w_s"] = _weights(gen, G, 2 * I, k)
        st["h_q"] = torch.empty((rows, I), dtype=torch.uint8, device=DEVICE)
        st["h_s"] = torch.empty((rows, I // BLOCK), device=DEVICE)
    return st


# ------------------------------------------------------------------ one pass

def _grouped_product(st):
    """fp32 [rows, n]: each row times its group's weights, the groups padded to
    the longest and multiplied as one batch."""
    off = st["grp_off"][0].long()
    rows = st["a_q"].shape[0]
    at = torch.arange(st["most"], device=DEVICE)
    row = (off[:-1, None] + at).clamp(max=rows - 1)  # [G, most]
    a = _dequant_rows(st["a_q"], st["a_s"])[row]
    p = torch.bmm(a, _dequant_weights(st["w_q"], st["w_s"]).transpose(1, 2))
    i = torch.arange(rows, device=DEVICE)
    g = torch.searchsorted(off[1:], i, right=True)
    return p[g, i - off[g]]


def _silu_mul(g, u):
    return g / (1 + torch.exp(-g)) * u


def _e4m3(q):
    return q.view(torch.float8_e4m3fn)


def _plain(st):
    op = st["case"]["op"]
    if op == "norm":
        v = st["x"].float()
        if st["res"] is not None:
            v = v + st["res"].float()
        y = v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * st["gamma"].float()
        out = {}
        if st["res"] is not None:
            out["res_out"] = v.bfloat16()
        if st["y"] is not None:
            out["y"] = y.bfloat16()
        if st["q"] is not None:
            q, out["s"] = _quant_rows(y)
            out["q"] = _e4m3(q)
        return out
    if op == "gemm":
        return _grouped_product(st).bfloat16()
    if op == "swiglu":
        g, u = _grouped_product(st).chunk(2, -1)
        q, s = _quant_rows(_silu_mul(g, u))
        return {"q": _e4m3(q), "s": s}
    # few: every (token, expert) pair with its expert's weights gathered
    T, R, H = st["case"]["T"], st["case"]["R"], st["case"]["H"]
    e = st["topk_idx"].long().flatten()
    x = _dequant_rows(*_quant_rows(st["x"].float())).repeat_interleave(R, 0)
    w13 = _dequant_weights(st["w13_q"][e], st["w13_s"][e])
    g, u = torch.bmm(w13, x.unsqueeze(-1)).squeeze(-1).chunk(2, -1)
    del w13
    h = _dequant_rows(*_quant_rows(_silu_mul(g, u)))
    y = torch.bmm(_dequant_weights(st["w2_q"][e], st["w2_s"][e]), h.unsqueeze(-1))
    return (y.view(T, R, H) * st["topk_w"][..., None]).sum(1).bfloat16()


def _own(st):
    from combine_expert_count_gb300 import moeroute as m
    shape, op = m.make_shape(*st["shape"]), st["case"]["op"]
    if op == "norm":
        m.moe_rmsnorm(shape, st["x"], st["gamma"], EPS, y=st["y"], q=st["q"], s=st["s"],
                      res=st["res"], res_out=st["res_out"])
        out = {n: st[n] for n in ("res_out", "y", "s") if st[n] is not None}
        if st["q"] is not None:
            out["q"] = _e4m3(st["q"])
        return out
    if op == "gemm":
        m.moe_expert_gemm(shape, st["case"]["n"], st["case"]["k"], st["a_q"], st["a_s"],
                          st["grp_off"], st["w_q"], st["w_s"], st["y"])
        return st["y"]
    if op == "swiglu":
        m.moe_expert_gemm_swiglu(shape, st["case"]["inter"], st["case"]["k"], st["a_q"],
                                 st["a_s"], st["grp_off"], st["w_q"], st["w_s"], st["h_q"],
                                 st["h_s"])
        return {"q": _e4m3(st["h_q"]), "s": st["h_s"]}
    m.moe_layer_few(shape, st["case"]["inter"], st["x"], st["topk_idx"], st["topk_w"],
                    st["w13_q"], st["w13_s"], st["w2_q"], st["w2_s"], st["h_q"], st["h_s"],
                    st["out"], st["status"])
    return st["out"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ cost

def work(case):
    if case["op"] == "norm":
        rows, H = case["rows"], case["H"]
        row = 2 * H + (4 * H if case["res"] else 0) + (2 * H if case["y"] else 0)
        row += H + H // 32 if case["q"] else 0
        return {"bytes": rows * row + 2 * H, "flops": 8 * rows * H}
    if case["op"] == "few":
        T, E, R, H, I = (case[c] for c in ("T", "E", "R", "H", "inter"))
        experts = E * (1 - (1 - R / E) ** T)  # expected, each token's R distinct
        weights = 3 * I * H * (1 + 4 / BLOCK**2)
        return {"bytes": experts * weights + T * (4 * H + 8 * R), "flops": 6 * T * R * I * H}
    rows, k = case["rows"], case["k"]
    n = case["n"] if case["op"] == "gemm" else 2 * case["inter"]
    groups = sum(m > 0 for m in _group_sizes(case))
    out = 2 * n if case["op"] == "gemm" else (n // 2) + (n // 2) // 32
    return {"bytes": rows * (k + k // 32 + out) + groups * n * k * (1 + 4 / BLOCK**2),
            "flops": 2 * rows * n * k}


# ------------------------------------------------------------------ 64 bits

def _values64(q):
    return q.view(torch.float8_e4m3fn).double()


def _blocks64(q, s):
    """Rows of e4m3 values, each times its block's scale."""
    return _values64(q) * s.double().repeat_interleave(BLOCK, -1)


def _weights64(q, s):
    s = s.double().repeat_interleave(BLOCK, -1).repeat_interleave(BLOCK, -2)
    return _values64(q) * s


def _round_e4m3(v):
    """The nearest e4m3 value of each |v| <= 448, ties to even, in 64 bits."""
    steps = torch.tensor([2.0**k for k in range(-9, 6)], dtype=torch.float64, device=v.device)
    _, exp = torch.frexp(v)
    step = steps[(exp - 4).clamp(min=-9).long() + 9]
    return torch.round(v / step) * step


def _quant64(v):
    """Codes and scales of rows; bf16 rows meet ties, which b * 448 / amax keeps."""
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    amax = b.abs().max(-1).values
    q = _round_e4m3(b * E4M3_MAX / torch.where(amax > 0, amax, torch.ones_like(amax))[..., None])
    return q.reshape(v.shape), amax / E4M3_MAX


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        out = {}
        v = st["x"].double()
        if case["res"]:
            v = v + st["res"].double()
            out["res_out"] = v
        y = v * (v.square().mean(-1, keepdim=True) + EPS).rsqrt() * st["gamma"].double()
        if case["y"]:
            out["y"] = y
        if case["q"]:
            out["q"], out["s"] = _quant64(y)
        return out
    if case["op"] == "few":
        T, R, H, I = (case[c] for c in ("T", "R", "H", "inter"))
        q, s = _quant64(st["x"].double())
        x = q * s.repeat_interleave(BLOCK, -1)
        out = torch.zeros((T, H), dtype=torch.float64, device=DEVICE)
        idx, w = st["topk_idx"].tolist(), st["topk_w"].double()
        for e in sorted({e for row in idx for e in row}):
            at = [(t, row.index(e)) for t, row in enumerate(idx) if e in row]
            t = torch.tensor([a[0] for a in at], device=DEVICE)
            k = torch.tensor([a[1] for a in at], device=DEVICE)
            p = x[t] @ _weights64(st["w13_q"][e], st["w13_s"][e]).T
            g, u = p[:, :I], p[:, I:]
            q, s = _quant64(g * torch.sigmoid(g) * u)
            h = q * s.repeat_interleave(BLOCK, -1)
            out[t] += w[t, k][:, None] * (h @ _weights64(st["w2_q"][e], st["w2_s"][e]).T)
        return out
    off = st["grp_off"][0].tolist()
    parts = []
    for g in range(case["G"]):
        a = slice(off[g], off[g + 1])
        parts.append(_blocks64(st["a_q"][a], st["a_s"][a])
                     @ _weights64(st["w_q"][g], st["w_s"][g]).T)
    p = torch.cat(parts)
    if case["op"] == "gemm":
        return p
    I = case["inter"]
    q, s = _quant64(p[:, :I] * torch.sigmoid(p[:, :I]) * p[:, I:])
    return {"q": q, "s": s}
