"""One token's vector through the int8 operators: what quant_rows_int8 gives of it, gemm_int8 takes."""
import pytest
import torch


@pytest.fixture(scope="module")
def far():
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    return far


def test_shapes_of_a_vector(far):
    """Without a GPU a vector gets as far as a matrix does; a vector of another length, or a scale with an axis, does not."""
    w, ws = torch.zeros(8, 256, dtype=torch.int8), torch.ones(8)
    q, s = torch.zeros(256, dtype=torch.int8), torch.tensor(1.0)
    with pytest.raises(ValueError, match="CUDA"):
        far.gemm_int8(q, s, w, ws)
    with pytest.raises(ValueError, match=r"\[n, k\]"):
        far.gemm_int8(q[:128], s, w, ws)
    with pytest.raises(ValueError, match=r"\[n, k\]"):
        far.gemm_int8(torch.tensor(1, dtype=torch.int8), s, w, ws)
    with pytest.raises(ValueError, match="x_scale"):
        far.gemm_int8(q, s[None], w, ws)


@pytest.mark.gpu
@pytest.mark.parametrize("k,n", [(264, 40), (4096, 1000), (1001, 7), (1040, 1)])
def test_a_vector_is_a_matrix_of_one_row(far, k, n):
    g = torch.Generator(device="cuda").manual_seed(k)
    wq, ws = far.quant_rows_int8(torch.randn(n, k, generator=g, device="cuda"))
    x, bias = torch.randn(k, generator=g, device="cuda").half(), torch.randn(n, generator=g, device="cuda").half()
    q, s = far.quant_rows_int8(x)
    want = far.gemm_int8(q[None], s[None], wq, ws, bias, out_dtype=torch.float16)
    assert s.shape == () and want.shape == (1, n)
    out = torch.empty(n, device="cuda", dtype=torch.float16)
    for y in (far.gemm_int8(q, s, wq, ws, bias, out_dtype=torch.float16),
              far.gemm_int8(q, s, wq, ws, bias, out_dtype=torch.float16, out=out),
              far.gemm_int8(q, s, wq, ws, bias, out_dtype=torch.float16, stream=torch.cuda.current_stream())):
        assert y.shape == (n,) and torch.equal(y, want[0])
    exact = ((q.double() @ wq.double().T).float() * (s * ws) + bias.float()).half()
    assert torch.equal(want[0], exact)
    empty = torch.empty(0, dtype=torch.int8, device="cuda")
    assert torch.equal(far.gemm_int8(empty, s, wq[:, :0], ws, bias, out_dtype=torch.float16), bias)
    assert far.device_status() == 0
