"""The gated feed-forward block at the ends of its numbers: activations below binary32's normal numbers, and the gradients'
operands, which are 16-bit values, at the ends of f16."""
import pytest
import torch

import ffn_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def far():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    return far


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("m", [40, None])
def test_activations_far_down(far, m, name):
    """gate from -4 to -128 in steps of 1/16 and finer, up = 2^100: act(gate) to 2^-15 of itself or 2^-143, and one rounding to bf16.
    (exp(-|z|) is off by at most 2^-150 where it is no normal number, times |gate| <= 104, where it ends: 2^-143.3.)"""
    t = torch.bfloat16
    g = -torch.arange(64, 2048, device="cuda") / 16.0
    g = g[torch.arange(0, g.numel(), max(1, g.numel() // m), device="cuda")[:m]] if m else g
    x = torch.zeros(g.numel(), 8, device="cuda", dtype=t)
    x[:, 0] = g.to(t)
    x[:, 1] = (g - x[:, 0].float()).to(t)
    x[:, 2] = 1
    assert bool((x[:, 0].double() + x[:, 1].double() == g.double()).all())
    wg, wu = (torch.zeros(16, 8, device="cuda", dtype=t) for _ in range(2))
    wg[:, :2], wu[:, 2] = 1, 2.0 ** 100
    out = far.gated_ffn(x, wg, wu, activation=name).double()
    a = ref.act(g.double(), name)[:, None]
    allowed = torch.maximum(2.0 ** -15 * a.abs(), torch.tensor(2.0 ** -143, device="cuda", dtype=torch.float64)) * 2.0 ** 100
    allowed = allowed * (1 + 2.0 ** -24) + ref.rounded(a.abs() * 2.0 ** 100 + allowed, t)
    assert bool(((out - a * 2.0 ** 100).abs() <= allowed).all()) and far.device_status() == 0


# dout, up, and what dout * up * act'(32) = dout * up is in f16
ENDS = [(2.0, 32752.0, 65504.0), (1.5, 43648.0, 65472.0), (1.5, 43680.0, float("inf")), (2.0, 32768.0, float("inf")),
        (-300.0, 300.0, -float("inf")), (2.0 ** -14, 2.0 ** -10, 2.0 ** -24), (2.0 ** -14, 2.0 ** -11, 0.0),
        (2.0 ** -14, 1.5 * 2.0 ** -11, 2.0 ** -24), (-(2.0 ** -24), 2.0 ** -24, -0.0)]


@pytest.mark.parametrize("m", [16, 300])
@pytest.mark.parametrize("dout,up,dgate", ENDS)
def test_gradients_at_the_ends_of_f16(far, m, dout, up, dgate):
    """dgate is rounded to f16 before the sums: from 65520 up it is infinite and up to 2^-25 zero, and so are the gradients, whatever
    the sums would have been; bf16 has binary32's range."""
    h, f = 24, 40
    x, wg, wu = torch.full((m, h), 2.0 ** -5), torch.full((f, h), 2.0 ** -8), torch.zeros(f, h)
    x, wg, wu = x.cuda().half(), wg.cuda().half(), wu.cuda().half()
    full = lambda v: torch.full((m, f), v, device="cuda").half()  # noqa: E731
    for name in ref.ACTS:
        dx, dwg, _ = far.gated_ffn_backward(full(dout), full(32.0), full(up), x, wg, wu, activation=name)
        # (f and m equal values: exact sums in binary32 where dgate is finite; 32 dout wu is 0)
        assert torch.equal(dx, torch.full_like(dx, torch.tensor(dgate * f * 2.0 ** -8).half().item()))
        assert torch.equal(dwg, torch.full_like(dwg, torch.tensor(dgate * m * 2.0 ** -5).half().item()))
    b = lambda v: v.bfloat16()  # noqa: E731
    dx, _, _ = far.gated_ffn_backward(b(full(dout)), b(full(32.0)), b(full(up)), b(x), b(wg), b(wu))
    exact = full(dout).bfloat16().double()[0, 0] * full(up).bfloat16().double()[0, 0]
    assert bool((dx.double() / (exact * f * 2.0 ** -8) - 1).abs().le(2.0 ** -7 + 2.0 ** -15).all()) and far.device_status() == 0
