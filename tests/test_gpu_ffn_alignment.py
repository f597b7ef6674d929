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


@pytest.mark.parametrize("m,h,f", [(9, 77, 333), (60, 72, 1001), (300, 264, 329), (300, 77, 334), (2000, 264, 1100), (2000, 520, 2743)])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
def test_rows_that_end_inside_16_bytes(far, t, m, h, f):
    """Aligned rows of wider matrices, of widths that are no multiple of 8: what lies behind the outputs' rows stays, and what
    lies behind the inputs' (NaN) does not count."""
    def rows(v):
        wide = torch.full((v.shape[0], (v.shape[1] + 7) // 8 * 8 + 8), float("nan"), device="cuda", dtype=t)
        return wide[:, :v.shape[1]].copy_(v)

    x, wg, wu = normal(m + f, t, (m, h), (f, h), (f, h))
    wg, wu = wg / h ** 0.5, wu / h ** 0.5
    x, wg, wu = rows(x), rows(wg), rows(wu)
    want = far.gated_ffn(x, wg, wu, save=True)
    assert all(bool(v.isfinite().all()) for v in want)
    for lefts in itertools.product((0, 8), (0, 1, 2), (0, 8)):
        outs, bigs = places(lefts, [(m, f)] * 3, t)
        far.gated_ffn(x, wg, wu, save=True, out=outs[0], gate_out=outs[1], up_out=outs[2])
        check(outs, bigs, want, lefts)
    dh, gate, up = (rows(v) for v in (normal(f, t, (m, f))[0], want[1], want[2]))
    space = torch.full((far.gated_ffn_backward_workspace_bytes(m, f),), 255, dtype=torch.uint8, device="cuda")
    want = far.gated_ffn_backward(dh, gate, up, x, wg, wu, workspace=space)
    assert all(bool(v.isfinite().all()) for v in want)
    for lefts in itertools.product((0, 8), (0, 1, 2), (0, 8)):
        outs, bigs = places(lefts, [(m, h), (f, h), (f, h)], t)
        far.gated_ffn_backward(dh, gate, up, x, wg, wu, dx=outs[0], dw_gate=outs[1], dw_up=outs[2])
        check(outs, bigs, want, lefts)
    assert far.device_status() == 0


@pytest.mark.parametrize("m,h,f", [(300, 264, 332), (2000, 264, 1100)])
def test_both_projections_in_one_buffer(far, m, h, f):
    """Halves of [tokens, 2 ffn]: the first on 16 bytes, the second 8 bytes off and right behind it."""
    x, wg, wu = normal(f, torch.bfloat16, (m, h), (f, h), (f, h))
    want = far.gated_ffn(x, wg, wu, save=True)
    both = torch.empty(m, 2 * f, device="cuda", dtype=torch.bfloat16)
    for first in (0, f):
        for _ in range(5):
            out, gate, up = far.gated_ffn(x, wg, wu, save=True, gate_out=both[:, first:first + f], up_out=both[:, f - first:2 * f - first])
            assert all(torch.equal(a, b) for a, b in zip((out, gate, up), want))
