"""gemm_int8 where its plan is CTA pairs (many rows), which every size here is asserted to take: exact integer sums bit for bit
at every height of tile, weights read as they stand and repacked, the largest sums, rare scales, strides and places,
workspaces that are not empty in graphs, on streams and in threads."""
import threading

import pytest
import torch
from test_gpu_int8 import TYPES, operands, product, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def far():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    return far


def pairs(far, m, n, k, rows=None):
    p = far.plan_gemm_int8(m, n, k)
    assert p["kind"] == 1 and rows in (None, p["rows"]), p
    return far.gemm_int8_workspace_bytes(m, n, k)


# (m, n, k, rows of x a tile): several sums of 1024 a tile, last blocks of 16 to 128, ragged last tiles either way
SIZES = [(400, 2500, 1040, 64), (130, 4100, 4112, 64), (260, 4100, 1040, 96), (1100, 1030, 1040, 96), (200, 8200, 1040, 128),
         (777, 2056, 2064, 128), (520, 4100, 1040, 160), (900, 2500, 1152, 160), (333, 8200, 1040, 192), (1500, 2056, 2064, 192),
         (3000, 512, 1024, 96), (2048, 2048, 1024, 128), (2100, 8200, 1040, 192), (4100, 4096, 512, None)]


@pytest.mark.parametrize("m,n,k,rows", SIZES)
def test_product(far, m, n, k, rows):
    pairs(far, m, n, k, rows)
    x, xs, w, ws = operands(m, n, k, m + n + k)
    for i, t in enumerate(TYPES.values()):
        bias = None if (m + i) % 2 else torch.randn(n, generator=rng(5), device="cuda").to(t)
        assert torch.equal(far.gemm_int8(x, xs, w, ws, bias, out_dtype=t), product(x, xs, w, ws, bias, t)), (t, far.device_status())
    assert far.device_status() == 0


@pytest.mark.parametrize("m,n,k", [(200, 520, 1100), (130, 8200, 1100), (777, 2056, 1101), (900, 2500, 1103), (333, 8200, 2059)])
def test_weights_repacked(far, m, n, k):
    """k that TMA cannot step over, and k that it can: rows of wt off 16 bytes, x alone off them, both."""
    pairs(far, m, n, k)
    x, xs, w, ws = operands(m, n, k, k)
    assert torch.equal(far.gemm_int8(x, xs, w, ws), product(x, xs, w, ws, None, torch.bfloat16))
    k = k // 16 * 16 + 16
    x, xs, w, ws = operands(max(m, 777), max(n, 2056), k, k, pad=13)
    pairs(far, *x.shape[:1], *w.shape)
    want = product(x, xs, w, ws, None, torch.float32)
    for a in (x, x.contiguous()):
        for b in (w, w.contiguous()):
            assert torch.equal(far.gemm_int8(a, xs, b, ws, out_dtype=torch.float32), want), (a.stride(), b.stride())
    assert far.device_status() == 0


@pytest.mark.parametrize("x0,w0", [(-128, -128), (127, -128), (127, 127), (-128, 127)])
@pytest.mark.parametrize("m,n,k", [(3000, 512, 1024), (777, 2056, 2048), (300, 4100, 16384), (300, 4100, 16380), (150, 8200, 131056),
                                   (150, 8200, 131071)])
def test_largest_sums(far, m, n, k, x0, w0):
    """Sums of 2^24 a 1024 values, 2^31 - 2^14 at the longest, and large sums that a few small products follow or precede."""
    pairs(far, m, n, k)
    x = torch.full((m, k), x0, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), w0, dtype=torch.int8, device="cuda")
    for first in (0, 128, n - 8):
        v = w[first:first + 8]
        v[1, k // 2:] = 1
        v[2, :k // 2] = -1
        v[3, ::2] = 0
        v[4, 1::2] = -v[4, 1::2].clamp(min=-127)
        v[5] = 0
        v[5, -1] = 1
        v[6, 1020:1024] = 3
        v[7, 1023] = 5
    x[m - 3, ::3] = 1
    x[m // 2, k - 20:] = -1
    one = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    y = far.gemm_int8(x, one[0], w, one[1], out_dtype=torch.float32)
    some = torch.tensor([0, 1, m // 2, m - 3, m - 1], device="cuda")  # the exact sums of every kind of row
    assert torch.equal(y[some], product(x[some], one[0][some], w, one[1], None, torch.float32))
    plain = torch.ones(m, dtype=torch.bool, device="cuda")
    plain[some] = False
    assert bool((y[plain] == y[0]).all()) and far.device_status() == 0


@pytest.mark.parametrize("m,n,k", [(3000, 512, 1024), (777, 2056, 2064)])
def test_scales(far, m, n, k):
    """Zero, far, infinite and NaN scales, in rows and columns of tiles whose other values keep their bits."""
    pairs(far, m, n, k)
    x, xs, w, ws = operands(m, n, k, 11)
    rare = torch.tensor([0.0, 1e30, 1e-30, float("inf"), float("nan"), 2.0 ** -149, 3e38, 2.0 ** -126], device="cuda")
    usual = product(x, xs, w, ws, None, torch.float32)
    ri, ci = torch.arange(8, device="cuda") * 37 + 5, torch.arange(8, device="cuda") * 61 + 3
    xs[ri], ws[ci] = rare, rare
    y = far.gemm_int8(x, xs, w, ws, out_dtype=torch.float32)
    rows, cols = torch.ones(m, dtype=torch.bool, device="cuda"), torch.ones(n, dtype=torch.bool, device="cuda")
    rows[ri], cols[ci] = False, False
    assert torch.equal(y[rows][:, cols], usual[rows][:, cols])
    acc = x.double() @ w.double().T
    want = (acc.float().double() * xs.double()[:, None] * ws.double()).float()
    fine = want.isfinite()
    assert bool((y[fine].double() - want[fine].double()).abs().le(2.0 ** -22 * want[fine].double().abs() + 2.0 ** -149).all())
    assert bool((y[~fine].isnan() | y[~fine].isinf()).all())
    assert bool((y[ri[0]][cols] == 0).all()) and bool((y[:, ci[0]][rows] == 0).all()) and bool(y[:, ci[4]].isnan().all())


@pytest.mark.parametrize("m,n,k", [(1100, 1030, 1040), (400, 2501, 1040), (200, 523, 1100)])
@pytest.mark.parametrize("t", TYPES)
def test_strides_and_places(far, m, n, k, t):
    """Rows of wider matrices on either side, an output inside a larger one at every alignment, leading axes, starts off 16."""
    pairs(far, m, n, k)
    x, xs, w, ws = operands(m, n, k, 3, pad=48)
    bias = torch.randn(n, generator=rng(7), device="cuda").to(TYPES[t])
    want = product(x, xs, w, ws, bias, TYPES[t])
    for left in (0, 1, 2, 8):
        big = torch.full((m + 2, (n + 7) // 8 * 8 + 16), 5.0, device="cuda").to(TYPES[t])
        out = big[1:m + 1, left:left + n]
        assert far.gemm_int8(x, xs, w, ws, bias, out_dtype=TYPES[t], out=out) is out
        assert torch.equal(out, want)
        out.fill_(5.0)
        assert bool((big == 5.0).all())
    y = far.gemm_int8(x.contiguous().view(2, m // 2, k), xs.view(2, m // 2), w, ws, bias, out_dtype=TYPES[t])
    assert y.shape == (2, m // 2, n) and torch.equal(y.view(m, n), want)
    odd = torch.empty(m * k + 3, dtype=torch.int8, device="cuda")[3:].view(m, k).copy_(x)
    odd_w = torch.empty(n * k + 5, dtype=torch.int8, device="cuda")[5:].view(n, k).copy_(w)
    assert torch.equal(far.gemm_int8(odd, xs, odd_w, ws, bias, out_dtype=TYPES[t]), want)


@pytest.mark.parametrize("m,n,k", [(3000, 512, 1024), (777, 2056, 2064), (200, 520, 1100)])
def test_streams_and_graphs(far, m, n, k):
    """A captured call replayed on new inputs, two graphs at once on two streams, explicit streams; a workspace given, full of
    another call's values, too small, off 16 bytes."""
    need = pairs(far, m, n, k)
    assert need > 0
    x, xs, w, ws = operands(m, n, k, 9)
    space = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    far.gemm_int8(x, xs, w, ws, out=out, workspace=space)
    assert bool((space[need:] == 255).all())
    graphs, outs = [], []
    for _ in range(2):
        outs.append(torch.zeros_like(out))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            far.gemm_int8(x, xs, w, ws, out=outs[-1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for seed in (1, 2):
        for a, b in zip((x, xs, w, ws), operands(m, n, k, seed)):
            a.copy_(b)
        want = product(x, xs, w, ws, None, torch.bfloat16)
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
        y = [far.gemm_int8(x, xs, w, ws, stream=s) for s in streams for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(v, want) for v in y)
        far.gemm_int8(x, xs, w, ws, out=out, workspace=space)
        assert torch.equal(out, want)
    for bad in (space[:16], space[:need - 1], space[8:need + 8]):
        with pytest.raises(far.FarError):
            far.gemm_int8(x, xs, w, ws, out=out, workspace=bad)
    assert far.device_status() == 0


def test_threads_on_their_own_streams(far):
    """Four threads, each with a stream, calling at once with the lock let go inside: every result its own."""
    sizes = [(3000, 512, 1024), (777, 2056, 2064), (200, 520, 1100), (1100, 1030, 1040)]
    assert all(pairs(far, *s) for s in sizes)
    cases = [operands(*s, s[0]) for s in sizes]
    want = [product(*c, None, torch.bfloat16) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = [far.gemm_int8(*cases[i]) for _ in range(30)]
        s.synchronize()
        if not all(torch.equal(g, want[i]) for g in got):
            wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and far.device_status() == 0
