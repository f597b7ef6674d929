"""Rows far below every value that matters: quant_rows_int8 takes what lies below 2^-100 as zero, the norm's int8 output only
what is zero.  From 2^-100 up they agree bit for bit."""
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

    return far


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [256, 1000])
def test_where_a_row_counts_as_zero(far, t, cols):
    """The norm of a row of +-1 is +-1 (eps 0): times a weight of 2^e for the row's size."""
    sign = torch.where(torch.rand(3, cols, generator=torch.Generator().manual_seed(1)) < 0.5, -1.0, 1.0).cuda().to(t)
    for e in (-90, -99, -100, -101, -110, -118):
        weight = torch.full((cols,), 2.0 ** e, device="cuda").to(t)
        out = far.rmsnorm(sign, weight, 0.0)
        assert bool((out == sign * weight).all())
        nq, ns = far.rmsnorm_quant(sign, weight, 0.0, "int8")
        q, s = far.quant_rows_int8(out)
        assert bool((ns == torch.tensor(2.0 ** e) / torch.tensor(127.0)).all()) and torch.equal(nq, (127 * sign.float()).to(torch.int8))
        if e >= -100:
            assert torch.equal(q, nq) and torch.equal(s, ns)
        else:
            assert bool((q == 0).all()) and bool((s == 0).all())
