"""Python's lock while a call of the native binding waits for the GPU's queue."""
import threading
import time

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


def calls(far):
    """Each entry point of the binding on a few values, its outputs given (so that the queue alone is waited for)."""
    b = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    x, w, y = b(1, 4, 64), torch.ones(64, device="cuda").bfloat16(), b(1, 4, 64)
    table, pos = far.rope_table(64, 64), torch.arange(1, device="cuda")
    ws = torch.empty(far.qk_backward_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    m, one, q, s = b(4, 128), torch.ones(128, device="cuda").bfloat16(), u(4, 128), torch.ones(4, 1, device="cuda")
    res, wq, wsc, out = b(4, 128), u(128, 128), torch.ones(1, 1, device="cuda"), b(4, 128)
    return {"rope": lambda: far.rope(x, None, table, pos, q_out=y),
            "qk_norm_rope": lambda: far.qk_norm_rope(x, None, w, None, 1e-6, table, pos, q_out=y),
            "qk_norm_rope_backward": lambda: far.qk_norm_rope_backward(x, None, x, None, w, None, 1e-6, table, pos, dq=y,
                                                                       workspace=ws),
            "rmsnorm_quant_block": lambda: far.rmsnorm_quant_block(m, one, 1e-6, q=q, scale=s),
            "fused_add_rmsnorm_quant_block": lambda: far.fused_add_rmsnorm_quant_block(m, res, one, 1e-6, q=q, scale=s,
                                                                                       residual_out=res),
            "quant_block_fp8": lambda: far.quant_block_fp8(m, q=q, scale=s),
            "gemm_fp8_block": lambda: far.gemm_fp8_block(q, s, wq, wsc, out=out)}


@pytest.mark.parametrize("name", ["rope", "qk_norm_rope", "qk_norm_rope_backward", "rmsnorm_quant_block",
                                  "fused_add_rmsnorm_quant_block", "quant_block_fp8", "gemm_fp8_block"])
def test_other_threads_run_while_a_call_waits(far, name):
    """The GPU is kept busy by one long kernel and its queue filled by small calls until one of them has to wait: meanwhile
    another Python thread goes on (its longest pause stays far below the wait)."""
    call = calls(far)[name]
    call()
    torch.cuda.synchronize()
    stop, pauses = threading.Event(), []

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            pauses.append(now - last)
            last = now

    other = threading.Thread(target=tick)
    other.start()
    waited = 0.0
    try:
        torch.cuda._sleep(1_000_000_000)  # about half a second
        for _ in range(20000):
            t = time.perf_counter()
            call()
            waited = max(waited, time.perf_counter() - t)
            if waited > 0.15:
                break
    finally:
        stop.set()
        other.join()
        torch.cuda.synchronize()
    if waited <= 0.15:
        pytest.skip("the queue took every call")
    assert max(pauses) < waited / 2, f"another thread stood still for {max(pauses):.3f} s of a call's {waited:.3f}"
