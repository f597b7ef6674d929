"""The per-head norm and rotation, and their gradients, from the definition in 64 bits, with
the error that binary32 steps may leave (the tests' tolerances).

Bounds, with u = 2^-24: a sum of D squares by fused multiply-adds in any tree of the kernels
(at most D/32 + 5 deep in the scalar kernel, V + 6 in the vector one; D/16 + 8 covers both)
is within (D/16 + 8) u of itself, and the root halves that.  The product by 1/D and the sum
with eps (3 u, halved), the reciprocal root (within two units in the last place: 4 u) and
the two products after it make 7.5 u more.  So n is within (D/32 + 12) u |n|, and a turned pair within that of |a c| + |b s|, plus 2 u of the same for
its two roundings.
"""
import torch

U = 2.0 ** -24
# half of each type's smallest step, where relative rounding ends
SMALLEST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def turn(x, cs, pairs, way=1.0):
    """x [..., D] turned by cs = (cos, sin) [tokens, 1, rot/2] (way -1: the transpose), and the
    same with absolute values throughout (the size of what was added)."""
    c, s = cs[0], way * cs[1]
    rot = 2 * c.shape[-1]
    if pairs == "half":
        ia = torch.arange(rot // 2, device=x.device)
        ib = ia + rot // 2
    else:
        ia = 2 * torch.arange(rot // 2, device=x.device)
        ib = ia + 1
    a, b = x[..., ia], x[..., ib]
    y, size = x.clone(), x.abs()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia], size[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, size


def rows_of(table, positions):
    half = table.shape[1] // 2
    r = table.double()[positions.clamp(0, table.shape[0] - 1).long()]
    return r[:, None, :half], r[:, None, half:]


def forward(x, w, eps, table, positions, pairs):
    """(y, allowed error) in 64 bits, for [tokens, heads, D]; w None: the rotation alone."""
    D = x.shape[-1]
    x = x.double()
    k = 2.0
    if w is not None:
        eps = float(torch.tensor(eps, dtype=torch.float32))
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
        k += D / 32 + 12
    y, size = turn(x, rows_of(table, positions), pairs)
    pad = (positions < 0)[:, None, None]
    return torch.where(pad, 0.0, y), torch.where(pad, 0.0, k * U * size)


def backward(dy, x, w, eps, table, positions, pairs):
    """(dx, its allowed error, dw, its allowed error).

    With g the turned gradient (within 3 u of its size), h = g w, u_ = x r: the mean of h u_ is
    within (D/16 + 8 + D/32 + 16) u of the mean of sizes, and r, u_ carry (D/32 + 12) u each.
    dw adds tokens x heads products, each within (D/32 + 16) u, one after another at worst."""
    T, H, D = x.shape
    eps = float(torch.tensor(eps, dtype=torch.float32))
    x, dy, w = x.double(), dy.double(), w.double()
    live = (positions >= 0)[:, None, None].double()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    n = x * r
    g, size = turn(dy, rows_of(table, positions), pairs, -1.0)
    h, hs = g * w, size * w.abs()
    dx = live * r * (h - n * (h * n).mean(-1, keepdim=True))
    ex = live * (D / 8 + 64) * U * r * (hs + n.abs() * (hs * n.abs()).mean(-1, keepdim=True))
    dw = (live * g * n).sum((0, 1))
    ew = (T * H + D / 32 + 24) * U * (live * size * n.abs()).sum((0, 1))
    return dx, ex, dw, ew


def within(got, ref, err, where=""):
    """got (its dtype's rounding of something within err of ref)."""
    t = got.dtype
    g = got.double()
    allowed = err + half_step(t) * (ref.abs() + err) + SMALLEST[t]
    off = (g - ref).abs()
    bad = ~(off <= allowed)
    assert not bad.any(), (f"{where}: {int(bad.sum())} of {bad.numel()} values off, worst "
                           f"{float((off / allowed).nan_to_num(1e30).max()):.3g} times what is allowed")
