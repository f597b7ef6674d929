"""The outputs of one call of the gated feed-forward block at alignments of their own: some leave the kernel by copies that
read a warp's box of shared memory later, others by the warp itself, in the same box.  Each mix gives the bits of the
contiguous call and touches nothing around its outputs."""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu
LEFT = (0, 2, 1)  # values before an output's rows: on 16, 4 and 2 bytes


@pytest.fixture(scope="module")
def far():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    return far


def normal(seed, t, *shapes):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(*s, generator=g, device="cuda").to(t) for s in shapes]


def places(lefts, shapes, t):
    """(outputs, the matrices that they lie in): rows a multiple of 16 bytes apart."""
    bigs = [torch.full((r + 2, (c + 7) // 8 * 8 + 16), 5.0, device="cuda", dtype=t) for r, c in shapes]
    return [b[1:r + 1, left:left + c] for b, left, (r, c) in zip(bigs, lefts, shapes)], bigs


def check(outs, bigs, want, lefts):
    for i, (o, b, w) in enumerate(zip(outs, bigs, want)):
        assert torch.equal(o, w), (i, lefts)
        o.fill_(5.0)
        assert bool((b == 5.0).all()), (i, lefts)


@pytest.mark.parametrize("m,h,f", [(300, 520, 328), (2000, 264, 1104), (2000, 520, 2744)])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
def test_forward(far, t, m, h, f):
    assert far.plan_gated_ffn(m, h, f)["kind"] == 1  # CTA pairs
    x, wg, wu = normal(m + f, t, (m, h), (f, h), (f, h))
    wg, wu = wg / h ** 0.5, wu / h ** 0.5
    want = far.gated_ffn(x, wg, wu, save=True)
    for lefts in itertools.product(LEFT, repeat=3):
        outs, bigs = places(lefts, [(m, f)] * 3, t)
        for _ in range(3):
            far.gated_ffn(x, wg, wu, save=True, out=outs[0], gate_out=outs[1], up_out=outs[2])
            check(outs, bigs, want, lefts)
    assert far.device_status() == 0


@pytest.mark.parametrize("m,h,f", [(300, 264, 200), (333, 1032, 2744), (70, 1032, 2744)])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
def test_backward(far, t, m, h, f):
    """Pairs that go from a tile of dw_gate on to one of dw_up, and single tiles."""
    dh, gate, up, x, wg, wu = normal(m + f, t, (m, f), (m, f), (m, f), (m, h), (f, h), (f, h))
    wg, wu = wg / h ** 0.5, wu / h ** 0.5
    want = far.gated_ffn_backward(dh, gate, up, x, wg, wu)
    for lefts in itertools.product(LEFT, repeat=3):
        outs, bigs = places(lefts, [(m, h), (f, h), (f, h)], t)
        for _ in range(3):
            far.gated_ffn_backward(dh, gate, up, x, wg, wu, dx=outs[0], dw_gate=outs[1], dw_up=outs[2])
            check(outs, bigs, want, lefts)
    assert far.device_status() == 0
