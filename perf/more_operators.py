"""What the 8-bit integer projection and the gated feed-forward block are measured on: the cases, their
inputs, the plain form of each operator in elementary torch operations, and its definition evaluated
in 64 bits.

    quant  a matrix quantised to int8 with a scale a row (a weight's output channels, activations' tokens)
    int8   the product of two such matrices: exact integer sums, scaled by token and channel, with a bias
    ffn    act(x @ w_gate^T) * (x @ w_up^T), both projections, the activation and the product at once
    back   its gradients, of x and of both weights
"""
import math

import torch

own = False

QMAX = 127.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("silu", "gelu", "gelu_tanh")


def listed():
    return [
        # a weight quantised once for serving, a scale for each output channel
        dict(name="quant weight", op="quant", rows=8192, cols=8192, type="bf16"),
        # the feed-forward block's inner values of a decode batch, on their way into an int8 projection
        dict(name="quant decode", op="quant", rows=48, cols=13312, type="f16"),
        # a decode batch through a projection: the weight's bytes alone count
        dict(name="int8 decode", op="int8", m=4, n=8192, k=8192, bias=False, type="bf16"),
        # a larger batch of single tokens through the feed-forward block's way back, long sums
        dict(name="int8 batch", op="int8", m=200, n=5120, k=13312, bias=True, type="f16"),
        # a ragged prompt, odd widths, binary32 out (logits)
        dict(name="int8 ragged", op="int8", m=777, n=2056, k=4112, bias=False, type="f32"),
        # a batch of prompts through a projection: the tensor cores' rate
        dict(name="int8 prompts", op="int8", m=16384, n=8192, k=8192, bias=True, type="bf16"),
        # one new token of a chat: both weights are read once
        dict(name="ffn one token", op="ffn", m=1, hidden=5120, ffn=13312, act="silu", save=False, type="bf16"),
        # a batch of single tokens of a smaller model, widths that fill no tile
        dict(name="ffn batch", op="ffn", m=60, hidden=2056, ffn=5640, act="gelu_tanh", save=False, type="f16"),
        # a batch of prompts
        dict(name="ffn prompts", op="ffn", m=8192, hidden=5120, ffn=13312, act="silu", save=False, type="bf16"),
        # a training step's way there on a ragged batch: both projections are kept for the way back
        dict(name="ffn training", op="ffn", m=4100, hidden=4096, ffn=8192, act="gelu", save=True, type="bf16"),
        # the way back of a training step
        dict(name="back training", op="back", m=8192, hidden=4096, ffn=8192, act="silu", type="bf16"),
        # the same on a few hundred tokens of a small model, odd widths
        dict(name="back small", op="back", m=333, hidden=1032, ffn=2744, act="gelu_tanh", type="f16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "int8", "int8", "ffn", "ffn", "back"])
    typ = rng.choice(["bf16", "f16"])
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192), type=rng.choice(["bf16", "f16", "f32"]))
    if op == "int8":
        return dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 128, 8192), k=16 * _log(rng, 8, 832), bias=rng.random() < 0.5,
                    type=rng.choice(["bf16", "f16", "f32"]))
    if op == "ffn":
        return dict(op=op, m=_log(rng, 1, 8192), hidden=8 * _log(rng, 32, 640), ffn=8 * _log(rng, 64, 1664),
                    act=rng.choice(ACTS), save=rng.random() < 0.4, type=typ)
    return dict(op=op, m=_log(rng, 16, 8192), hidden=8 * _log(rng, 32, 512), ffn=8 * _log(rng, 64, 1024), act=rng.choice(ACTS),
                type=typ)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _quantise(x):
    """int8 codes and scales of a binary32 matrix, a row at a time: scale = amax / 127, code = round(x * (127 / amax))."""
    amax = x.abs().amax(-1)
    top = torch.full_like(amax, QMAX)
    zero = amax == 0
    scale = torch.where(zero, 0.0, amax / top)
    inv = torch.where(zero, 0.0, top / amax)
    return torch.round(x * inv[:, None]).clamp(-QMAX, QMAX).to(torch.int8), scale


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    op, t = case["op"], TYPES[case["type"]]
    s = {"case": dict(case)}
    if op == "quant":
        # rows of sizes of their own, as tokens and channels have
        s["x"] = (normal(case["rows"], case["cols"]) * torch.exp(normal(case["rows"], 1))).to(t)
    elif op == "int8":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"], s["xs"] = _quantise(normal(m, k) * torch.exp(normal(m, 1)))
        s["w"], s["ws"] = _quantise(normal(n, k) * torch.exp(0.3 * normal(n, 1)) / math.sqrt(k))
        s["bias"] = normal(n).to(t) if case["bias"] else None
    else:
        m, h, f = case["m"], case["hidden"], case["ffn"]
        # behind a norm: values of about one; weights that keep that size
        s |= {"x": normal(m, h).to(t), "wg": (normal(f, h) / math.sqrt(h)).to(t), "wu": (normal(f, h) / math.sqrt(h)).to(t)}
        if op == "back":
            row = torch.exp(0.3 * normal(m, 1))
            s |= {"gate": (1.5 * row * normal(m, f)).to(t), "up": (row * normal(m, f)).to(t), "dh": normal(m, f).to(t)}
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

_C = math.sqrt(2.0 / math.pi)
_A = 0.044715


def _activation(g, act):
    """(act(g), act'(g)) in binary32."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        c = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    th = torch.tanh(_C * (g + _A * g * g * g))
    return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * _C * (1.0 + 3.0 * _A * g * g)


def run(state):
    s, case = state, state["case"]
    op, t = case["op"], TYPES[case["type"]]
    if own:
        import mixed_precision_residual_gb300 as far
        if op == "quant":
            return far.quant_rows_int8(s["x"])
        if op == "int8":
            return far.gemm_int8(s["x"], s["xs"], s["w"], s["ws"], s["bias"], out_dtype=t)
        if op == "ffn":
            return far.gated_ffn(s["x"], s["wg"], s["wu"], activation=case["act"], save=case["save"])
        return far.gated_ffn_backward(s["dh"], s["gate"], s["up"], s["x"], s["wg"], s["wu"], activation=case["act"])
    if op == "quant":
        return _quantise(s["x"].float())
    if op == "int8":
        y = (s["x"].float() @ s["w"].float().t()) * s["xs"][:, None] * s["ws"]
        return (y if s["bias"] is None else y + s["bias"].float()).to(t)
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    if op == "ffn":
        gate, up = x @ wg.t(), x @ wu.t()
        h = (_activation(gate, case["act"])[0] * up).to(t)
        return (h, gate.to(t), up.to(t)) if case["save"] else h
    dh = s["dh"].float()
    a, slope = _activation(s["gate"].float(), case["act"])
    dgate, dup = dh * s["up"].float() * slope, dh * a
    return (dgate @ wg + dup @ wu).to(t), (dgate.t() @ x).to(t), (dup.t() @ x).to(t)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, b = case["op"], SIZE[case["type"]]
    if op == "quant":
        r, c = case["rows"], case["cols"]
        return {"bytes": r * c * (b + 1) + 4 * r, "flops": 3 * r * c}
    if op == "int8":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + m * n * b + (n * b if case["bias"] else 0), "flops": 2 * m * n * k}
    m, h, f = case["m"], case["hidden"], case["ffn"]
    if op == "ffn":
        return {"bytes": b * (m * h + 2 * f * h + m * f * (3 if case["save"] else 1)), "flops": 4 * m * h * f}
    # dh, gate, up, x and the weights in; the gradients of x and of the weights out
    return {"bytes": b * (3 * m * f + 2 * m * h + 4 * f * h), "flops": 8 * m * h * f}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _gated64(g, u, act):
    if act == "silu":
        return u * g * torch.special.expit(g)
    if act == "gelu":
        return u * g * torch.special.ndtr(g)
    return u * g * torch.special.expit(2.0 * _C * (g + _A * g ** 3))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        # the contract's steps, each in 64 bits and rounded to binary32 where the contract says so
        x = s["x"].double()
        amax = x.abs().max(1, keepdim=True).values
        live = amax > 0
        inv = torch.where(live, QMAX / amax, 0.0).float().double()
        return torch.round((x * inv).float().double()).to(torch.int8), (amax / QMAX).squeeze(1)
    if op == "int8":
        y = torch.einsum("mk,nk->mn", s["x"].double() * s["xs"].double()[:, None], s["w"].double() * s["ws"].double()[:, None])
        return y if s["bias"] is None else y + s["bias"].double()
    x, wg, wu = (s[n].double() for n in ("x", "wg", "wu"))
    if op == "ffn":
        gate, up = torch.einsum("mh,fh->mf", x, wg), torch.einsum("mh,fh->mf", x, wu)
        h = _gated64(gate, up, case["act"])
        return (h, gate, up) if case["save"] else h
    leaves = [s[n].double().requires_grad_() for n in ("gate", "up")]
    dgate, dup = torch.autograd.grad(_gated64(*leaves, case["act"]), leaves, s["dh"].double())
    return (torch.einsum("mf,fh->mh", dgate, wg) + torch.einsum("mf,fh->mh", dup, wu), torch.einsum("mf,mh->fh", dgate, x),
            torch.einsum("mf,mh->fh", dup, x))
