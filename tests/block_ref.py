"""128-block FP8 quantisation and the block-scaled product from their definitions, in 64 bits on
the CPU; quantisation is exact (every step is one correctly rounded operation)."""
import torch

BLOCK, QMAX, TINY = 128, 448.0, 2.0 ** -100


def nblocks(n):
    return -(-n // BLOCK)


def e4m3(v):
    """The nearest E4M3 value (ties to even, saturated) of a float64 tensor; NaN stays NaN."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp(min=-9))
    r = (torch.round(v / step) * step).clamp(-QMAX, QMAX)
    return torch.where(v.isinf(), torch.sign(v) * QMAX, r)


def spread(s, r, c, rows):
    """One scale a value from scales a block (rows: 1 or 128 of them share one)."""
    s = s.repeat_interleave(BLOCK, 1)[:, :c]
    return (s.repeat_interleave(BLOCK, 0) if rows == BLOCK else s)[:r]


def quantise(x, block):
    """(values of the codes, scales) of a matrix, as float64 / float32: scale = fl32(amax / 448),
    value = E4M3(fl32(x * fl32(448 / amax))); amax below 2^-100 counts as zero."""
    x = x.double()
    r, c = x.shape
    rows = BLOCK if block == "tile" else 1
    pr, pc = -(-r // rows) * rows, nblocks(c) * BLOCK
    p = torch.nn.functional.pad(x, (0, pc - c, 0, pr - r)).view(pr // rows, rows, pc // BLOCK, BLOCK)
    a = p.abs()
    amax = torch.where(a.isnan().any(3).any(1), torch.nan, a.nan_to_num(0.0, posinf=float("inf")).amax((1, 3)))
    zero = amax < TINY
    scale = torch.where(zero, 0.0, amax / QMAX).float()
    inv = torch.where(zero, 0.0, QMAX / amax).float()
    v = (x * spread(inv.double(), r, c, rows)).float().double()
    return e4m3(v), scale


def same_values(codes, values):
    """FP8 codes against values, NaN equal to NaN (zeros of either sign equal)."""
    v = codes.view(torch.float8_e4m3fn).float().double().cpu()
    values = values.cpu()
    return bool(((v == values) | (v.isnan() & values.isnan())).all())


def same_scales(a, b):
    a, b = a.cpu(), b.cpu()
    return a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())


def product(xq, xs, wq, ws):
    """(product, allowed binary32 error) of block-scaled matrices, float64.

    A block's sum of up to 128 exact products, and the sum of the blocks, in binary32 with
    every addition rounded or truncated: (128 + blocks) additions of at most 2^-22 of the sum
    of magnitudes each, and three products by scales of 2^-24."""
    m, k = xq.shape
    n = wq.shape[0]
    rows = 1 if ws.shape[0] == n else BLOCK
    x = xq.view(torch.float8_e4m3fn).double() * spread(xs.double(), m, k, 1)
    w = wq.view(torch.float8_e4m3fn).double() * spread(ws.double(), n, k, rows)
    y, size = x @ w.T, x.abs() @ w.abs().T
    return y, (min(k, BLOCK) + nblocks(k) + 4) * 2.0 ** -22 * size
