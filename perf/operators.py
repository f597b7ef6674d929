"""What the per-head norm and rotation, the 128-block FP8 quantisation and the block-scaled
FP8 product are measured on: the cases, their inputs, the plain form of each operator in
elementary torch operations, and its definition evaluated in 64 bits.

    qk     per-head RMSNorm of queries and keys with the position rotation in the same pass
    rope   the rotation alone (interleaved pairs, part of the head)
    qkback the gradients of qk: of q, k and of the two norm weights
    norm   residual add + RMSNorm with a 128-block FP8 (E4M3) output
    quant  a matrix quantised to FP8 in rows of 128 or 128 x 128 tiles, as it stands or transposed
    gemm   the product of two block-scaled FP8 matrices
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
BLOCK = 128
QMAX = 448.0
TINY = 2.0 ** -100  # a block whose largest magnitude is below this is stored as zeros, scale 0
POSITIONS = 32768   # rows of the rotation table
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one new token of a chat: latency alone
        dict(name="qk one token", op="qk", tokens=1, heads=32, kv=8, dim=128, rot=128, pairs="half", type="bf16"),
        # a batch of packed prompts, q and k read from the packed projection
        dict(name="qk prompts", op="qk", tokens=16384, heads=32, kv=8, dim=128, rot=128, pairs="half", type="bf16"),
        # rotation without a norm, a third of each head in interleaved pairs, an odd token count
        dict(name="rope part of head", op="rope", tokens=2049, heads=16, kv=16, dim=192, rot=64, pairs="inter", type="f16"),
        # a training step's way back through the same norm and rotation
        dict(name="qk backward", op="qkback", tokens=8192, heads=32, kv=8, dim=128, rot=128, pairs="half", type="bf16"),
        # the same in binary32 on a small ragged batch, heads of 80
        dict(name="qk backward f32", op="qkback", tokens=777, heads=12, kv=12, dim=80, rot=80, pairs="half", type="f32"),
        # the norm ahead of an FP8 projection: a decode batch, and a batch of prompts
        dict(name="norm decode", op="norm", tokens=8, hidden=2048, type="bf16", weight="bf16"),
        dict(name="norm prompts", op="norm", tokens=16384, hidden=5120, type="bf16", weight="bf16"),
        # a weight quantised once for serving: 128 x 128 tiles
        dict(name="quant weight", op="quant", rows=8192, cols=8192, block="tile", transpose=False, type="bf16"),
        # a gradient quantised along the tokens for the weight's gradient: read by rows, written transposed
        dict(name="quant transposed", op="quant", rows=2064, cols=5120, block="row", transpose=True, type="f16"),
        # a decode batch through a projection: the weight's bytes alone count
        dict(name="gemm decode", op="gemm", m=4, n=8192, k=8192, scales="tile", type="bf16"),
        # a weight's gradient: both operands scaled by rows of 128 tokens, a ragged token count, binary32 out
        dict(name="gemm gradient", op="gemm", m=5120, n=2056, k=4112, scales="row", type="f32"),
        # a batch of prompts through a projection: the tensor cores' rate
        dict(name="gemm prompts", op="gemm", m=16384, n=8192, k=8192, scales="tile", type="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "rope", "qkback", "norm", "quant", "gemm", "gemm"])
    typ = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("qk", "rope", "qkback"):
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        return dict(op=op, tokens=_log(rng, 1, 16384 if op != "qkback" else 8192), heads=kv * rng.choice([1, 2, 4]), kv=kv,
                    dim=dim, rot=rng.choice([dim, dim, dim // 2 // 16 * 16]), pairs=rng.choice(["half", "inter"]), type=typ)
    if op == "norm":
        weight = typ if rng.random() < 0.7 else "f32"
        return dict(op=op, tokens=_log(rng, 1, 8192), hidden=8 * _log(rng, 32, 1024), type=typ, weight=weight)
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192), block=rng.choice(["row", "tile"]),
                    transpose=rng.random() < 0.5, type=typ)
    return dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 128, 8192), k=16 * _log(rng, 8, 512),
                scales=rng.choice(["tile", "tile", "row"]), type=typ)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _table(rot, dev):
    """cos and sin of position x frequency, in binary32 from binary64 angles: [positions, cos | sin]."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    angle = torch.arange(POSITIONS, dtype=torch.float64, device=dev)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def _positions(tokens, g, dev):
    """Packed sequences of different lengths, each from a start of its own."""
    cuts = torch.randint(0, max(tokens, 1), (max(1, tokens // 700),), generator=g, device=dev)
    flag = torch.zeros(tokens, dtype=torch.int64, device=dev)
    flag[cuts] = 1
    flag[0] = 1
    seq = flag.cumsum(0) - 1
    first = torch.nonzero(flag).flatten()
    start = torch.randint(0, POSITIONS - tokens, (first.numel(),), generator=g, device=dev)
    return torch.arange(tokens, device=dev) - first[seq] + start[seq]


def _blocks(x, block):
    """x with its last axis cut in blocks of 128 (row) or both axes in tiles: padded with zeros to whole blocks."""
    r, c = x.shape
    pc = -(-c // BLOCK) * BLOCK
    pr = -(-r // BLOCK) * BLOCK if block == "tile" else r
    return torch.nn.functional.pad(x, (0, pc - c, 0, pr - r))


def _quantise(x, block):
    """FP8 codes and scales of a binary32 matrix: scale = amax / 448, code = E4M3(x * (448 / amax))."""
    r, c = x.shape
    p = _blocks(x, block)
    b = p.view(r, -1, BLOCK) if block == "row" else p.view(p.shape[0] // BLOCK, BLOCK, -1, BLOCK)
    amax = b.abs().amax(-1) if block == "row" else b.abs().amax((1, 3))
    top = torch.full_like(amax, QMAX)
    zero = amax < TINY
    scale = torch.where(zero, 0.0, amax / top)
    inv = torch.where(zero, 0.0, top / amax)
    v = b * (inv[..., None] if block == "row" else inv[:, None, :, None])
    return v.clamp(-QMAX, QMAX).view_as(p)[:r, :c].to(E4M3), scale


def _spread(scale, block, r, c):
    """A matrix's scales, one for each element."""
    s = scale.repeat_interleave(BLOCK, 1)[:, :c]
    return s if block == "row" else s.repeat_interleave(BLOCK, 0)[:r]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    op, t = case["op"], TYPES[case["type"]]
    s = {"case": dict(case)}
    if op in ("qk", "rope", "qkback"):
        n, h, k, d = case["tokens"], case["heads"], case["kv"], case["dim"]
        # the packed projection's output: queries, keys, values, each head with a size of its own
        qkv = (normal(n, h + 2 * k, d) * torch.exp(normal(1, h + 2 * k, 1))).to(t)
        s |= {"q": qkv[:, :h], "k": qkv[:, h:h + k], "positions": _positions(n, g, dev), "table": _table(case["rot"], dev)}
        if op != "rope":
            s |= {"qw": (1 + 0.1 * normal(d)).to(t), "kw": (1 + 0.1 * normal(d)).to(t), "eps": 1e-6}
        if op == "qkback":
            s |= {"dq": normal(n, h, d).to(t), "dk": normal(n, k, d).to(t)}
    elif op == "norm":
        n, h = case["tokens"], case["hidden"]
        row = torch.exp(torch.empty(n, 1, device=dev).uniform_(math.log(0.01), math.log(100.0), generator=g))
        s |= {"x": (normal(n, h) * row).to(t), "residual": (normal(n, h) * row).to(t),
              "weight": (1 + 0.1 * normal(h)).to(TYPES[case["weight"]]), "eps": 1e-6}
    elif op == "quant":
        s |= {"x": (normal(case["rows"], case["cols"]) * torch.exp(normal(case["rows"], 1))).to(t)}
    else:
        x = normal(case["m"], case["k"]) * torch.exp(normal(case["m"], 1))
        w = normal(case["n"], case["k"]) * 0.02
        s["x"], s["xs"] = _quantise(x, "row")
        s["w"], s["ws"] = _quantise(w, case["scales"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _rotate(x, table, positions, rot, pairs, way=1.0):
    """The rotation of the first `rot` values of each head (way -1: its transpose), binary32."""
    cs = table[positions][:, None, :]
    c, sn = cs[..., :rot // 2], way * cs[..., rot // 2:]
    if pairs == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * c - b * sn, b * c + a * sn, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2), x[..., rot:]], -1)


def _plain_qk(x, w, s, case):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
    return _rotate(x, s["table"], s["positions"], case["rot"], case["pairs"])


def _plain_qk_back(dy, x, w, s, case):
    x, t = x.float(), x.dtype
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
    n = x * r
    gr = _rotate(dy.float(), s["table"], s["positions"], case["rot"], case["pairs"], -1.0)
    dw = (gr * n).double().sum((0, 1)).float()
    h = gr * w.float()
    return (r * (h - n * (h * n).mean(-1, keepdim=True))).to(t), dw


def _plain_norm(s):
    """The rounding contract of fused_add_rmsnorm, then 128-block quantisation of the values `out` would have: the
    roundings to the weight's and the output's type are the operator's own, everything else is binary32."""
    t, wt = s["x"].dtype, s["weight"].dtype
    out_t = torch.promote_types(t, wt)
    v = s["x"].float() + s["residual"].float()
    total = (v * v).double().sum(-1, keepdim=True).float()
    var = total / torch.full_like(total, v.shape[1])
    rstd = torch.ones_like(var) / torch.sqrt(var + s["eps"])
    out = ((v * rstd).to(wt).float() * s["weight"].float()).to(out_t).float()
    q, scale = _quantise(out, "row")
    return q, scale, v.to(t)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import mixed_precision_residual_gb300 as far
        inter = case.get("pairs") == "inter"
        if op == "qk":
            return far.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"], s["positions"], interleaved=inter)
        if op == "rope":
            return far.rope(s["q"], s["k"], s["table"], s["positions"], interleaved=inter)
        if op == "qkback":
            return far.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"],
                                             s["positions"], interleaved=inter)
        if op == "norm":
            return far.fused_add_rmsnorm_quant_block(s["x"], s["residual"], s["weight"], s["eps"])
        if op == "quant":
            return far.quant_block_fp8(s["x"], block=case["block"], transpose=case["transpose"])
        return far.gemm_fp8_block(s["x"], s["xs"], s["w"], s["ws"], out_dtype=TYPES[case["type"]])
    t = TYPES[case["type"]]
    if op == "qk":
        return tuple(_plain_qk(s[x], s[x + "w"], s, case).to(t) for x in ("q", "k"))
    if op == "rope":
        return tuple(_rotate(s[x].float(), s["table"], s["positions"], case["rot"], case["pairs"]).to(t) for x in ("q", "k"))
    if op == "qkback":
        dq, dqw = _plain_qk_back(s["dq"], s["q"], s["qw"], s, case)
        dk, dkw = _plain_qk_back(s["dk"], s["k"], s["kw"], s, case)
        return dq, dk, dqw, dkw
    if op == "norm":
        return _plain_norm(s)
    if op == "quant":
        x = s["x"].float()
        return _quantise(x.t().contiguous() if case["transpose"] else x, case["block"])
    m, n, k = case["m"], case["n"], case["k"]
    x = s["x"].float() * _spread(s["xs"], "row", m, k)
    w = s["w"].float() * _spread(s["ws"], case["scales"], n, k)
    return (x @ w.t()).to(t)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("qk", "rope", "qkback"):
        n = case["tokens"]
        values = n * (case["heads"] + case["kv"]) * case["dim"]
        per = (3 if op == "qkback" else 2) * SIZE[case["type"]]
        # the positions, and one row of the table for each token
        return {"bytes": values * per + n * (8 + 4 * case["rot"]), "flops": values * {"qk": 7, "rope": 3, "qkback": 14}[op]}
    if op == "norm":
        n, h = case["tokens"], case["hidden"]
        return {"bytes": n * h * (3 * SIZE[case["type"]] + 1) + n * -(-h // BLOCK) * 4 + h * SIZE[case["weight"]], "flops": 8 * n * h}
    if op == "quant":
        r, c = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"], case["cols"])
        scales = -(-c // BLOCK) * (r if case["block"] == "row" else -(-r // BLOCK))
        return {"bytes": r * c * (SIZE[case["type"]] + 1) + 4 * scales, "flops": 3 * r * c}
    m, n, k = case["m"], case["n"], case["k"]
    kb = -(-k // BLOCK)
    scales = m * kb + (n if case["scales"] == "row" else -(-n // BLOCK)) * kb
    return {"bytes": m * k + n * k + 4 * scales + m * n * SIZE[case["type"]], "flops": 2 * m * n * k}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _turn(x, s, case):
    """Complex numbers turned by the table's angles: the definition of the rotation."""
    rot = case["rot"]
    row = s["table"].double().index_select(0, s["positions"])
    z = torch.complex(row[:, :rot // 2], row[:, rot // 2:])[:, None, :]
    if case["pairs"] == "half":
        y = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * z
        head = torch.cat([y.real, y.imag], -1)
    else:
        head = torch.view_as_real(torch.view_as_complex(x[..., :rot].reshape(*x.shape[:2], rot // 2, 2)) * z).flatten(-2)
    return torch.cat([head, x[..., rot:]], -1)


def _forward64(x, w, s, case):
    if w is not None:
        x = w * x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"])
    return _turn(x, s, case)


def _e4m3(v):
    """The nearest E4M3 value, ties to even, saturated: 3 bits behind the leading one, none below 2^-9."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp(min=-9))
    return (torch.round(v / step) * step).clamp(-QMAX, QMAX)


def _blocks64(v, block):
    """Codes' values and scales of a matrix of binary32 values held in 64 bits, block after block by scatter."""
    r, c = v.shape
    i = torch.arange(r, device=v.device)[:, None] // (1 if block == "row" else BLOCK)
    j = torch.arange(c, device=v.device)[None, :] // BLOCK
    wide = -(-c // BLOCK)
    flat = (i * wide + j).expand(r, c).reshape(-1)
    amax = torch.zeros(int(flat[-1]) + 1, dtype=torch.float64, device=v.device)
    amax = amax.scatter_reduce(0, flat, v.abs().reshape(-1), "amax")
    live = amax >= TINY
    scale = torch.where(live, amax / QMAX, 0.0).float()
    inv = torch.where(live, QMAX / amax.clamp(min=TINY), 0.0).float().double()
    q = _e4m3((v.reshape(-1) * inv[flat]).float().double()).view(r, c)
    return q, scale.double().view(-1, wide)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "qk":
        return tuple(_forward64(s[x].double(), s[x + "w"].double(), s, case) for x in ("q", "k"))
    if op == "rope":
        return tuple(_forward64(s[x].double(), None, s, case) for x in ("q", "k"))
    if op == "qkback":
        leaves = [s[x].double().requires_grad_() for x in ("q", "k", "qw", "kw")]
        q, k, qw, kw = leaves
        y = (_forward64(q, qw, s, case) * s["dq"].double()).sum() + (_forward64(k, kw, s, case) * s["dk"].double()).sum()
        return tuple(torch.autograd.grad(y, leaves))
    if op == "norm":
        # the contract's steps, each in 64 bits and rounded to binary32 where the contract says so
        t, wt = s["x"].dtype, s["weight"].dtype
        f32 = lambda v: v.float().double()  # noqa: E731
        v = f32(s["x"].double() + s["residual"].double())
        var = f32(f32(f32(v ** 2).sum(1)) / v.shape[1])
        rstd = f32(1.0 / f32(torch.sqrt(f32(var + torch.tensor(s["eps"], dtype=torch.float32, device=v.device).double()))))
        n = f32(v * rstd[:, None]).to(wt).double()
        out = f32(n * s["weight"].double()).to(torch.promote_types(t, wt)).double()
        q, scale = _blocks64(out, "row")
        return q, scale, v.to(t).double()
    if op == "quant":
        x = s["x"].double()
        return _blocks64(x.t() if case["transpose"] else x, case["block"])
    # block by block along k: exact integers of E4M3 products, scaled once a block
    m, n, k = case["m"], case["n"], case["k"]
    x, w = s["x"].double(), s["w"].double()
    y = torch.zeros(m, n, dtype=torch.float64, device=x.device)
    rows = torch.arange(n, device=x.device) // (1 if case["scales"] == "row" else BLOCK)
    for b in range(-(-k // BLOCK)):
        cut = slice(b * BLOCK, min(k, (b + 1) * BLOCK))
        y.addmm_(x[:, cut] * s["xs"][:, b, None].double(), (w[:, cut] * s["ws"][rows, b, None].double()).t())
    return y
