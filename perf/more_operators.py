"""What the operators around the experts of a block are measured on.

Four operators that stand next to the exchange in a mixture-of-experts block:
the product of bf16 rows and weights with bias, activation and residual in its
epilogue (``linear``: a router's logits, a projection, a shared expert's second
product), the two projections of a gated feed-forward with the activation and
the product between them (``glu``: a shared expert's first half), the router's
choice (``topk``: the dispatch's ids and weights from logits), and the end of a
block (``block``: a norm after the branch, its gate and scale, the residual and
the next block's norm with its 8-bit coding).  Sizes are those of this
repository's configurations (hidden 7168 with 256 experts, hidden 2048 with 128
experts, top-8, expert widths of 2048 and 768), and odd ones.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
BLOCK = 128
E4M3_MAX = 448.0
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token through a shared expert's second product, onto the routed experts' output
        dict(name="linear_one", op="linear", rows=1, n=7168, k=2048, act="none", bias=False,
             res=True, f32=False),
        # router logits of a decode step of 16 ranks x 128 tokens, kept in 32 bits
        dict(name="linear_router", op="linear", rows=2048, n=256, k=7168, act="none", bias=False,
             res=False, f32=True),
        # a projection back to the residual stream, a batch of odd size
        dict(name="linear_batch", op="linear", rows=509, n=7168, k=7168, act="none", bias=True,
             res=True, f32=False),
        # the same over a prompt, with an activation
        dict(name="linear_prefill", op="linear", rows=8191, n=7168, k=7168, act="gelu_tanh",
             bias=True, res=True, f32=False),
        # one token through a shared expert's first half
        dict(name="glu_one", op="glu", rows=1, inter=2048, k=7168, act="silu", bias=False),
        # a few sequences' decode step, hidden 2048
        dict(name="glu_decode", op="glu", rows=61, inter=768, k=2048, act="gelu", bias=True),
        # a shared expert's first half over a prompt
        dict(name="glu_prefill", op="glu", rows=8191, inter=2048, k=7168, act="silu", bias=False),
        # decode step: sigmoid scores with a correction bias, four of eight groups kept
        dict(name="topk_decode", op="topk", rows=2048, E=256, R=8, score="sigmoid", bias=True,
             groups=8, kept=4, best=2, renorm=True, scale=2.5, off=0, coarse=False),
        # a prompt's tokens: softmax scores renormalised over the chosen
        dict(name="topk_prefill", op="topk", rows=32767, E=128, R=8, score="softmax", bias=False,
             groups=1, kept=1, best=1, renorm=True, scale=1.0, off=0, coarse=False),
        # one token's row at the end of a block while decoding
        dict(name="block_one", op="block", rows=1, H=7168, post=True, gates=1, scale=0.5, res=True,
             y=True, q=True),
        # a decode step of 16 ranks x 128 tokens, a gate row for each rank's sequence
        dict(name="block_decode", op="block", rows=2048, H=7168, post=True, gates=16, scale=1.0,
             res=True, y=True, q=False),
        # a prompt's tokens, bf16 for the router and 8 bits for the products; odd count
        dict(name="block_prefill", op="block", rows=32767, H=7168, post=True, gates=1, scale=1.0,
             res=True, y=True, q=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("linear", "glu", "topk", "block"))
    if op == "linear":
        return dict(op=op, rows=_log(rng, 1, 8191), n=_log(rng, 1, 7168), k=8 * _log(rng, 1, 896),
                    act=rng.choice(ACTS), bias=rng.random() < 0.5, res=rng.random() < 0.5,
                    f32=rng.random() < 0.3)
    if op == "glu":
        return dict(op=op, rows=_log(rng, 1, 8191), inter=_log(rng, 1, 2048),
                    k=8 * _log(rng, 1, 896), act=rng.choice(ACTS), bias=rng.random() < 0.5)
    if op == "topk":
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * _log(rng, 2, 1024 // groups)
        kept = rng.randint(1, groups)
        c = dict(op=op, rows=_log(rng, 1, 32767), E=E, R=rng.randint(1, min(32, E * kept // groups)),
                 score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5, groups=groups,
                 kept=kept, best=rng.randint(1, 2), renorm=rng.random() < 0.7,
                 scale=rng.choice((1.0, 2.5)), coarse=rng.random() < 0.3)
        c["off"] = rng.choice((0, 0, rng.randint(0, E - 1)))
        return c
    rows, q = _log(rng, 1, 32767), rng.random() < 0.6
    gates = rng.choice((0, 1, rows, rng.choice([d for d in range(1, 65) if rows % d == 0])))
    return dict(op=op, rows=rows, H=BLOCK * _log(rng, 1, 56), post=rng.random() < 0.7, gates=gates,
                scale=rng.choice((1.0, 0.5, 0.22)), res=rng.random() < 0.8,
                y=not q or rng.random() < 0.7, q=q)


# ------------------------------------------------------------------ inputs

def _rows(gen, rows, k):
    """Activations with a few channels several times larger than the others."""
    x = torch.randn((rows, k), generator=gen, device=DEVICE)
    return x * (1 + 7 * (torch.rand(k, generator=gen, device=DEVICE) < 0.01))


def _weights(gen, n, k):
    return (torch.randn((n, k), generator=gen, device=DEVICE) / math.sqrt(k)).bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    st, rows = dict(case=case), case["rows"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEVICE)

    if case["op"] in ("linear", "glu"):
        k, glu = case["k"], case["op"] == "glu"
        n = case["inter"] if glu else case["n"]
        outs = 2 * n if glu else n
        st["x"], st["w"] = _rows(gen, rows, k).bfloat16(), _weights(gen, outs, k)
        st["bias"] = (0.3 * randn(outs)).bfloat16() if case["bias"] else None
        f32 = not glu and case["f32"]
        st["res"] = randn(rows, n).bfloat16() if not glu and case["res"] else None
        st["y"] = torch.empty((rows, n), dtype=torch.float32 if f32 else torch.bfloat16,
                              device=DEVICE)
        st["shape"] = (1, rows, 1, 1, BLOCK, 0)
        return st
    if case["op"] == "topk":
        E = case["E"]
        logits = 1.5 * randn(rows, E) + 0.5 * randn(E)  # some experts are liked more
        if case["coarse"]:  # logits that came through 16 bits: many are equal
            logits = logits.bfloat16().float()
        if case["off"]:  # experts that are out of service
            logits[:, torch.randperm(E, generator=gen, device=DEVICE)[:case["off"]]] = -math.inf
        st["logits"] = logits
        st["bias"] = 0.1 * randn(E) if case["bias"] else None
        st["idx"] = torch.empty((rows, case["R"]), dtype=torch.int32, device=DEVICE)
        st["w"] = torch.empty((rows, case["R"]), device=DEVICE)
        st["shape"] = (1, rows, E, case["R"], BLOCK, 0)
        return st
    H = case["H"]
    st["x"] = _rows(gen, rows, H).bfloat16()
    st["res"] = (3 * _rows(gen, rows, H)).bfloat16() if case["res"] else None
    st["gamma"] = (1 + 0.2 * randn(H)).bfloat16()
    st["post"] = (1 + 0.2 * randn(H)).bfloat16() if case["post"] else None
    st["gate"] = (0.7 * randn(case["gates"], H)).bfloat16() if case["gates"] else None
    st["res_out"] = torch.empty_like(st["x"])
    st["y"] = torch.empty_like(st["x"]) if case["y"] else None
    st["q"] = torch.empty((rows, H), dtype=torch.uint8, device=DEVICE) if case["q"] else None
    st["s"] = torch.empty((rows, H // BLOCK), device=DEVICE) if case["q"] else None
    st["shape"] = (1, rows, 1, 1, H, 0)
    return st


# ------------------------------------------------------------------ one pass

def _act(name, v):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    return v


def _quant_rows(v):
    """fp32 [..., k] -> e4m3 values and scales amax/448 (0 for a zero block)."""
    b = v.unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1)
    s = amax / torch.full_like(amax, E4M3_MAX)  # by a tensor: a number becomes its reciprocal
    q = torch.where(s[..., None] > 0, b / s[..., None], torch.zeros_like(b))
    return q.to(torch.float8_e4m3fn).flatten(-2), s


def _first(v, n):
    """The places of the n largest of each row, equal ones by their order."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[..., :n]


def _plain_topk(st):
    c, l = st["case"], st["logits"]
    shifted = l.double() - l.double().amax(-1, keepdim=True)
    if c["score"] == "softmax":
        wide = torch.exp(shifted)
        wide = wide / wide.sum(-1, keepdim=True)
        e = torch.exp(shifted.float())
        score = e / e.sum(-1, keepdim=True)
    else:
        wide = 1 / (1 + torch.exp(-l.double()))
        score = 1 / (1 + torch.exp(-l))
    gone = torch.full_like(wide, -math.inf)
    # the values that choose, in 64 bits: two that are near each other are still in order
    choice = l.double() if st["bias"] is None else wide + st["bias"].double()
    choice = torch.where(l == -math.inf, gone, choice)
    if c["groups"] > 1:
        g = choice if c["best"] == 1 or st["bias"] is not None else torch.where(
            l == -math.inf, gone, wide)
        g = g.unflatten(-1, (c["groups"], -1))
        best = torch.sort(g, dim=-1, descending=True).values[..., :c["best"]]
        kept = _first(best.sum(-1), c["kept"])
        on = torch.zeros(best.shape[:-1], dtype=torch.bool, device=DEVICE).scatter_(-1, kept, True)
        choice = torch.where(on.repeat_interleave(c["E"] // c["groups"], -1), choice, gone)
        # an expert of a group that was not kept is behind the masked ones of those that were
        order = _first(on.repeat_interleave(c["E"] // c["groups"], -1).double(), c["E"])
        place = _first(choice.gather(-1, order), c["R"])
        idx = order.gather(-1, place)
    else:
        idx = _first(choice, c["R"])
    w = score.gather(-1, idx)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return {"idx": idx.int(), "w": w * c["scale"]}


def _plain(st):
    c = st["case"]
    if c["op"] in ("linear", "glu"):
        p = st["x"].float() @ st["w"].float().T
        if st["bias"] is not None:
            p = p + st["bias"].float()
        if c["op"] == "glu":
            g, u = p.chunk(2, -1)
            return (_act(c["act"], g) * u).bfloat16()
        p = _act(c["act"], p)
        if st["res"] is not None:
            p = p + st["res"].float()
        return p if c["f32"] else p.bfloat16()
    if c["op"] == "topk":
        return _plain_topk(st)
    b = st["x"].float()
    if st["post"] is not None:
        b = b / torch.sqrt((b * b).mean(-1, keepdim=True) + EPS) * st["post"].float()
    if st["gate"] is not None:
        b = (b.unflatten(0, (c["gates"], -1)) * st["gate"].float()[:, None]).flatten(0, 1)
    v = b * c["scale"]
    if st["res"] is not None:
        v = v + st["res"].float()
    out = {"res_out": v.bfloat16()}
    y = v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * st["gamma"].float()
    if c["y"]:
        out["y"] = y.bfloat16()
    if c["q"]:
        out["q"], out["s"] = _quant_rows(y)
    return out


def _own(st):
    from combine_expert_count_gb300 import moeroute as m
    shape, c = m.make_shape(*st["shape"]), st["case"]
    if c["op"] == "linear":
        m.moe_linear(shape, c["n"], c["k"], st["x"], st["w"], st["y"], bias=st["bias"],
                     res=st["res"], act=c["act"])
        return st["y"]
    if c["op"] == "glu":
        m.moe_linear_glu(shape, c["inter"], c["k"], st["x"], st["w"], st["y"], bias=st["bias"],
                         act=c["act"])
        return st["y"]
    if c["op"] == "topk":
        m.moe_topk(shape, st["logits"], st["idx"], st["w"], bias=st["bias"], score=c["score"],
                   groups=c["groups"], kept=c["kept"], best=c["best"], renorm=c["renorm"],
                   scale=c["scale"])
        return {"idx": st["idx"], "w": st["w"]}
    m.moe_block_norm(shape, st["x"], st["gamma"], EPS, res_out=st["res_out"], y=st["y"],
                     q=st["q"], s=st["s"], post_gamma=st["post"], gate=st["gate"],
                     gates=c["gates"], scale=c["scale"], res=st["res"])
    out = {n: st[n] for n in ("res_out", "y", "s") if st[n] is not None}
    if c["q"]:
        out["q"] = st["q"].view(torch.float8_e4m3fn)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ cost

def work(case):
    rows = case["rows"]
    if case["op"] in ("linear", "glu"):
        k, glu = case["k"], case["op"] == "glu"
        n = case["inter"] if glu else case["n"]
        outs = 2 * n if glu else n
        out = 4 if not glu and case["f32"] else 2
        res = 2 if not glu and case["res"] else 0
        return {"bytes": 2 * (rows + outs) * k + (2 * outs if case["bias"] else 0)
                + rows * n * (out + res), "flops": 2 * rows * outs * k}
    if case["op"] == "topk":
        E, R = case["E"], case["R"]
        return {"bytes": rows * (4 * E + 8 * R) + (4 * E if case["bias"] else 0),
                "flops": rows * E * 8}
    H = case["H"]
    row = 4 * H + (2 * H if case["res"] else 0) + (2 * H if case["y"] else 0)
    row += H + H // 32 if case["q"] else 0
    vectors = 1 + case["post"] + case["gates"]
    return {"bytes": rows * row + 2 * H * vectors, "flops": 14 * rows * H}


# ------------------------------------------------------------------ 64 bits

def _act64(name, v):
    if name == "relu":
        return v.clamp(min=0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * torch.special.erfc(-v / 2 ** 0.5) / 2
    if name == "gelu_tanh":  # (1 + tanh z) / 2 = sigmoid(2 z)
        return v * torch.sigmoid((8 / math.pi) ** 0.5 * v * (1 + 0.044715 * v.square()))
    return torch.sigmoid(v) if name == "sigmoid" else v


def _round_e4m3(v):
    """The nearest e4m3 value of each |v| <= 448, ties to even, in 64 bits."""
    _, exp = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (exp - 4).clamp(min=-9))
    return torch.round(v / step) * step


def _exact_topk(st):
    """Row by row on the host would be slow: each row's order is found by counting how
    many experts come before each."""
    c, l = st["case"], st["logits"].double()
    E, R, per = c["E"], c["R"], c["E"] // c["groups"]
    if c["rows"] * E * E > 2 ** 31:
        return None
    b = torch.zeros(E, dtype=torch.float64, device=DEVICE) if st["bias"] is None \
        else st["bias"].double()
    score = torch.softmax(l, -1) if c["score"] == "softmax" else torch.sigmoid(l)
    out = l == -math.inf
    key = torch.where(out, l, score + b if st["bias"] is not None else l)
    at = torch.arange(E, device=DEVICE)

    def before(v):  # [rows, n]: how many of the row come before each
        n = v.shape[-1]
        a, z = v[:, None, :], v[:, :, None]
        return ((a > z) | ((a == z) & (at[:n][None, None] < at[:n][None, :, None]))).sum(-1)
    if c["groups"] > 1:
        worth = key if c["best"] == 1 or st["bias"] is not None else torch.where(out, l, score)
        worth = worth.reshape(-1, c["groups"], per).topk(min(c["best"], per), -1).values.sum(-1)
        kept = (before(worth) < c["kept"]).repeat_interleave(per, -1)
    else:
        kept = torch.ones_like(out)
    # kept ones first, each lot by its key and place
    level = torch.where(kept, before(key), before(key) + E)
    order = level.argsort(-1)[:, :R]
    w = score.gather(-1, order)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    return {"idx": order.int(), "w": w * c["scale"]}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("linear", "glu"):
        p = st["x"].double().matmul(st["w"].double().t())
        if case["bias"]:
            p += st["bias"].double()
        if case["op"] == "glu":
            n = case["inter"]
            return _act64(case["act"], p[:, :n]) * p[:, n:]
        p = _act64(case["act"], p)
        return p + st["res"].double() if case["res"] else p
    if case["op"] == "topk":
        return _exact_topk(st)
    rows = case["rows"]
    v = st["x"].double()
    if case["post"]:
        v = v * (v.square().mean(-1, keepdim=True) + EPS).rsqrt() * st["post"].double()
    if case["gates"]:
        which = torch.arange(rows, device=DEVICE) // (rows // case["gates"])
        v = v * st["gate"].double()[which]
    v = v * case["scale"]
    if case["res"]:
        v = v + st["res"].double()
    out = {"res_out": v}
    y = v * (v.square().mean(-1, keepdim=True) + EPS).rsqrt() * st["gamma"].double()
    if case["y"]:
        out["y"] = y
    if case["q"]:
        b = y.reshape(rows, -1, BLOCK)
        amax = b.abs().amax(-1)
        safe = torch.where(amax > 0, amax, torch.ones_like(amax))[..., None]
        out["q"] = _round_e4m3(b * E4M3_MAX / safe).reshape(rows, -1)
        out["s"] = amax / E4M3_MAX
    return out
