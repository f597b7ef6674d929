"""Long back-to-back chains of the int8 product and the gated feed-forward block over one set of buffers: each kernel
overwrites what an earlier one read and reads what the one ahead of it wrote, with every launch a programmatic
dependent one.  The same chain of plain launches, where no kernel starts before the one ahead has finished, gives
the bits to match."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def far():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    yield far
    far.set_programmatic_launch(True)


def same_under_both(far, chain, times=3):
    try:
        far.set_programmatic_launch(False)
        want = chain()
        far.set_programmatic_launch(True)
        for _ in range(times):
            for i, (a, b) in enumerate(zip(chain(), want)):
                assert torch.equal(a, b), f"link {i} differs under programmatic launch"
    finally:
        far.set_programmatic_launch(True)
    assert far.device_status() == 0 and bool(want.isfinite().all()) and bool((want[-1] != 0).any())


@pytest.mark.parametrize("m,k", [(4, 512), (60, 1024), (130, 512), (600, 1024), (1100, 2048), (600, 1032), (700, 1001)])
def test_quantise_and_multiply(far, m, k):
    """x -> codes of x, codes of one of three weights into the same place, their product into x, over and over: few rows, a
    cluster's rows, CTA pairs (whose weight is written just ahead), and weights that TMA cannot read as they stand."""
    g = torch.Generator(device="cuda").manual_seed(m + k)
    weights = [(torch.randn(k, k, generator=g, device="cuda") / k ** 0.5).bfloat16() for _ in range(3)]
    start = torch.randn(m, k, generator=g, device="cuda").bfloat16()
    space = torch.empty(far.gemm_int8_workspace_bytes(m, k, k) + 16, dtype=torch.uint8, device="cuda")
    xq, xs = torch.empty(m, k, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    wq, ws = torch.empty(k, k, dtype=torch.int8, device="cuda"), torch.empty(k, device="cuda")

    def chain():
        x, seen = start.clone(), torch.zeros(40, m, k, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        for i in range(40):
            far.quant_rows_int8(x, xq, xs)
            far.quant_rows_int8(weights[i % 3], wq, ws)
            far.gemm_int8(xq, xs, wq, ws, out=x, workspace=space)
            far.gemm_int8(xq, xs, wq, ws, out=seen[i], workspace=space)
        torch.cuda.synchronize()
        return seen

    same_under_both(far, chain)


@pytest.mark.parametrize("m,h", [(4, 512), (60, 520), (130, 512), (600, 512)])
def test_there_and_back(far, m, h):
    """x -> the block's values and both projections into the same places, their gradients, of which dx, normalised, is the next
    x; the weights of three pairs in turn are copied into the same place, from which the weights' gradients are added to them."""
    g = torch.Generator(device="cuda").manual_seed(m + h)
    f, t = 2 * h, torch.bfloat16

    def n(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(t)

    start, pairs, one = n(m, h), [(n(f, h) / h ** 0.5, n(f, h) / h ** 0.5) for _ in range(3)], torch.ones(h, device="cuda").to(t)
    wg, wu = torch.empty(f, h, dtype=t, device="cuda"), torch.empty(f, h, dtype=t, device="cuda")
    space = torch.empty(far.gated_ffn_backward_workspace_bytes(m, f), dtype=torch.uint8, device="cuda")
    out, gate, up = (torch.empty(m, f, dtype=t, device="cuda") for _ in range(3))
    dx, dwg, dwu = torch.empty_like(start), torch.empty_like(wg), torch.empty_like(wu)
    row = torch.ones(f, 1, device="cuda").to(t) / 64

    def chain():
        x = start.clone()
        seen = torch.zeros(40, m + 2 * f, h, dtype=t, device="cuda")
        torch.cuda.synchronize()
        for i in range(40):
            torch.add(pairs[i % 3][0], dwg * row if i else 0, out=wg)
            torch.add(pairs[i % 3][1], dwu * row if i else 0, out=wu)
            far.gated_ffn(x, wg, wu, save=True, out=out, gate_out=gate, up_out=up)
            far.gated_ffn_backward(out, gate, up, x, wg, wu, dx=dx, dw_gate=dwg, dw_up=dwu, workspace=space)
            far.rmsnorm(dx, one, 1e-6, out=x)
            far.rmsnorm(dwg, one, 1e-6, out=dwg)
            far.rmsnorm(dwu, one, 1e-6, out=dwu)
            seen[i, :m], seen[i, m:m + f], seen[i, m + f:] = x, dwg, dwu
        torch.cuda.synchronize()
        return seen

    same_under_both(far, chain)
