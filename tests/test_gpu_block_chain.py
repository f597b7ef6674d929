"""A long back-to-back chain of the block-quantised operators over one set of buffers: each kernel overwrites what
an earlier one read and reads what the one ahead of it wrote, with every launch a programmatic dependent one.  The
same chain of plain launches, where no kernel starts before the one ahead has finished, gives the bits to match."""
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


def chain(far, m, k, block, norm, links):
    """x -> codes and scales of x, codes and scales of one of three weights, their product into x, over and over."""
    g = torch.Generator(device="cuda").manual_seed(m + k)
    x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
    weights = [(torch.randn(k, k, generator=g, device="cuda") * torch.exp(torch.randn(k, 1, generator=g, device="cuda")) /
                k ** 0.5).bfloat16() for _ in range(3)]
    one = torch.ones(k, device="cuda").bfloat16()
    kb = -(-k // 128)
    xq, xs = torch.empty(m, k, dtype=torch.uint8, device="cuda"), torch.empty(m, kb, device="cuda")
    wq = torch.empty(k, k, dtype=torch.uint8, device="cuda")
    ws = torch.empty(k if block == "row" else kb, kb, device="cuda")
    seen = torch.zeros(links, m, k, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    for i in range(links):
        if norm or i % 2 == 0:  # the values shrink or grow by the weights' sizes: normalised at every or every other link
            far.rmsnorm_quant_block(x, one, 1e-6, q=xq, scale=xs)
        else:
            far.quant_block_fp8(x, q=xq, scale=xs)
        far.quant_block_fp8(weights[i % 3], block, q=wq, scale=ws)
        far.gemm_fp8_block(xq, xs, wq, ws, out=x)
        far.gemm_fp8_block(xq, xs, wq, ws, out=seen[i])
    torch.cuda.synchronize()
    assert far.device_status() == 0
    return seen


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("block", ["tile", "row"])
@pytest.mark.parametrize("m,k", [(4, 512), (40, 1024), (300, 512), (700, 1024), (30, 520)])
def test_chain_over_the_same_buffers(far, m, k, block, norm):
    """Few rows, several rows a CTA, CTA pairs, and k that takes the plain kernel (520: scales of five blocks)."""
    links = 60
    try:
        far.set_programmatic_launch(False)
        want = chain(far, m, k, block, norm, links)
        far.set_programmatic_launch(True)
        for _ in range(3):
            got = chain(far, m, k, block, norm, links)
            for i in range(links):
                assert torch.equal(got[i], want[i]), f"link {i} differs under programmatic launch"
    finally:
        far.set_programmatic_launch(True)
    assert bool(want.isfinite().all()) and bool((want[-1] != 0).any())
