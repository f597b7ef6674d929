"""The block-scaled FP8 product into slices of wider matrices: every output dtype at every width modulo 16 bytes, on and off
16-byte rows.  The values are the contiguous call's, and nothing around the slice is touched: a TMA copy writes whole
16-byte units, so the last ones of rows that end inside one may not leave that way."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def far():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    return far


@pytest.mark.parametrize("m", [7, 60, 1000])
@pytest.mark.parametrize("block", ["tile", "row"])
@pytest.mark.parametrize("t", TYPES)
def test_product_in_a_wider_matrix(far, t, block, m):
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, 512, generator=g, device="cuda").bfloat16()
    xq, xs = far.quant_block_fp8(x)
    for n in (1, 3, 31, 33, 64, 95, 130, 520, 521, 522, 523, 524, 525, 526, 527, 1990):
        w = torch.randn(n, 512, generator=g, device="cuda").bfloat16()
        wq, ws = far.quant_block_fp8(w, block=block)
        want = far.gemm_fp8_block(xq, xs, wq, ws, out_dtype=TYPES[t])
        for left in (0, 8, 1, 2):
            big = torch.full((m + 2, (n + 7) // 8 * 8 + 16), 5.0, device="cuda", dtype=TYPES[t])
            out = big[1:m + 1, left:left + n]
            assert far.gemm_fp8_block(xq, xs, wq, ws, out_dtype=TYPES[t], out=out) is out
            assert torch.equal(out, want), (n, left)
            out.fill_(5.0)
            assert bool((big == 5.0).all()), (n, left)
    assert far.device_status() == 0
