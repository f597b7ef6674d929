"""The gated feed-forward block from its formulas in 64 bits, with the error that binary32 sums, the
activations' 2^-15 and one rounding to 16 bits allow.

A sum of k exact products, every addition rounded or truncated: each off by at most 2^-22 of the sum
of the magnitudes.  An activation's slope is at most 1.13 (gelu: 1.129, silu: 1.100) in magnitude."""
import math

import torch

SLOPE = 1.13
FUNCTION = 2.0 ** -15
ACTS = ("silu", "gelu", "gelu_tanh")
C, A = math.sqrt(2.0 / math.pi), 0.044715


def half_step(t):
    """(relative half step, half of the smallest number)."""
    return torch.finfo(t).eps / 2, torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def rounded(size, t):
    r, least = half_step(t)
    return r * size + least


def phi(g):
    """The normal distribution, to full relative precision (torch.special.ndtr on the GPU is 0 from -9.2 down)."""
    return 0.5 * torch.erfc(-g * math.sqrt(0.5))


def act(g, name):
    if name == "silu":
        return g * torch.special.expit(g)
    if name == "gelu":
        return g * phi(g)
    return g * torch.special.expit(2 * C * (g + A * g ** 3))  # (1 + tanh(y)) / 2, without cancellation


def slope(g, name):
    if name == "silu":
        return torch.special.expit(g) * (1 + g * torch.special.expit(-g))
    if name == "gelu":
        return phi(g) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    y = 2 * C * (g + A * g ** 3)
    return torch.special.expit(y) * (1 + g * torch.special.expit(-y) * 2 * C * (1 + 3 * A * g * g))


def forward(x, wg, wu, name):
    """[(value, allowed error)] of out, gate and up."""
    t, k = x.dtype, x.shape[1]
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, u = x @ wg.T, x @ wu.T
    step = (k + 1) * 2.0 ** -22
    eg, eu = step * (x.abs() @ wg.abs().T), step * (x.abs() @ wu.abs().T)
    a = act(g, name)
    h = a * u
    eh = (SLOPE * eg + FUNCTION * (a.abs() + SLOPE * eg)) * (u.abs() + eu) + a.abs() * eu
    eh = eh + 2.0 ** -23 * (h.abs() + eh)
    return [(v, e + rounded(v.abs() + e, t)) for v, e in ((h, eh), (g, eg), (u, eu))]


def backward(dh, gate, up, x, wg, wu, name):
    """[(value, allowed error)] of dx, dw_gate and dw_up: dgate and dup are rounded to 16 bits on the way."""
    t = x.dtype
    dh, gate, up, x, wg, wu = (v.double() for v in (dh, gate, up, x, wg, wu))
    dg, du = dh * up * slope(gate, name), dh * act(gate, name)
    # the slope's two terms are at most 1 and about 1/2 in magnitude, each right to 2^-15; a few binary32 products
    eg = (dh * up).abs() * 1.5 * FUNCTION + 2.0 ** -22 * dg.abs()
    eu = du.abs() * (FUNCTION + 2.0 ** -22)
    eg, eu = eg + rounded(dg.abs() + eg, t), eu + rounded(du.abs() + eu, t)
    ag, au, ax = dg.abs() + eg, du.abs() + eu, x.abs()
    dx, dwg, dwu = dg @ wg + du @ wu, dg.T @ x, du.T @ x
    ex = eg @ wg.abs() + eu @ wu.abs() + (2 * wg.shape[0] + 2) * 2.0 ** -22 * (ag @ wg.abs() + au @ wu.abs())
    step = (x.shape[0] + 1) * 2.0 ** -22
    egw, euw = eg.T @ ax + step * (ag.T @ ax), eu.T @ ax + step * (au.T @ ax)
    return [(v, e + rounded(v.abs() + e, t)) for v, e in ((dx, ex), (dwg, egw), (dwu, euw))]


def within(got, want, allowed):
    d = (got.double() - want).abs()
    return bool(torch.isfinite(got).all()) and bool((d <= allowed).all())
