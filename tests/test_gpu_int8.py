"""int8 with a scale a row on the GPU: quantising against the formula in binary32, the product against exact
integer sums and the contract's binary32 operations, both bit for bit; strides, places outputs must not
touch, streams and graphs."""
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


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def quantised(x):
    """(codes, scales) on the CPU: every step one correctly rounded binary32 operation."""
    x = x.cpu().float()
    amax = x.abs().amax(-1) if x.shape[-1] else x.new_zeros(x.shape[:-1])
    amax = torch.where(x.isnan().any(-1), torch.nan, amax)
    zero = amax < 2.0 ** -100
    top = torch.full_like(amax, 127.0)
    scale = torch.where(zero, 0.0, amax / top)
    inv = torch.where(zero, 0.0, top / amax)
    q = torch.where(amax.isfinite()[..., None], torch.round(x * inv[..., None]), 0.0)
    return q.to(torch.int8), scale


def same(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


# one warp to 16 warps a row, 8 chunks a thread, and longer; lengths of no whole chunk
COLS = [0, 1, 7, 8, 24, 128, 264, 1000, 1024, 1032, 2056, 4096, 5120, 8192, 13312, 16384, 16392, 32768, 32776, 40000]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("t", TYPES)
def test_quant(far, t, cols):
    for rows in (1, 5, 33):
        g = rng(cols + rows)
        x = (torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(3 * torch.randn(rows, 1, generator=g, device="cuda"))).to(TYPES[t])
        q, s = far.quant_rows_int8(x)
        qr, sr = quantised(x)
        assert torch.equal(q.cpu(), qr) and torch.equal(s.cpu(), sr)
    assert far.device_status() == 0


@pytest.mark.parametrize("cols", [5, 512, 40000])
@pytest.mark.parametrize("t", TYPES)
def test_quant_special_rows(far, t, cols):
    """Zero, tiny, huge and non-finite rows; ties; the largest value at either end."""
    x = torch.randn(12, cols, generator=rng(1), device="cuda")
    x[0] = 0
    x[1] *= 0
    x[1, -1] = torch.finfo(TYPES[t]).tiny
    x[2, 0] = float("nan")
    x[3, -1] = float("inf")
    x[4, 0] = -float("inf")
    x[5] = torch.finfo(TYPES[t]).max
    x[6] = -127.0
    x[6, 0] = 63.5
    x[7] = 0.5
    x[7, -1] = 127.0
    x[8] = 2.0 ** -101
    x[9] = 2.0 ** -100
    x = x.to(TYPES[t])
    q, s = far.quant_rows_int8(x)
    qr, sr = quantised(x)
    assert torch.equal(q.cpu(), qr) and same(s.cpu(), sr)
    assert int(q.min()) >= -127


def test_quant_places(far):
    """Strided rows, leading axes, outputs given and what lies around them, a misaligned start."""
    g = rng(3)
    wide = torch.randn(40, 700, generator=g, device="cuda").half()
    for x in (wide[:, 8:520], wide[:, 3:300], wide[::2, :64], wide.view(4, 10, 700)):
        q, s = far.quant_rows_int8(x)
        qr, sr = quantised(x)
        assert q.shape == x.shape and torch.equal(q.cpu(), qr) and torch.equal(s.cpu(), sr)
    buf, sc = torch.full((42 * 700,), 99, dtype=torch.int8, device="cuda"), torch.full((42,), 7.0, device="cuda")
    q, s = buf[700:41 * 700].view(40, 700), sc[1:41]
    assert far.quant_rows_int8(wide, q, s)[0] is q
    qr, sr = quantised(wide)
    assert torch.equal(q.cpu(), qr) and torch.equal(s.cpu(), sr)
    assert bool((buf[:700] == 99).all()) and bool((buf[41 * 700:] == 99).all()) and float(sc[0]) == 7 and float(sc[41]) == 7


def test_quant_of_one_row(far):
    """A vector has one scale, without an axis."""
    x = torch.randn(264, generator=rng(8), device="cuda").half()
    q, s = far.quant_rows_int8(x)
    qr, sr = quantised(x)
    assert q.shape == (264,) and s.shape == () and torch.equal(q.cpu(), qr) and torch.equal(s.cpu(), sr)


def product(x, xs, w, ws, bias, t):
    """The contract: the exact integer rounded to binary32, the scales' product, the bias, one rounding."""
    acc = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    for k in range(0, x.shape[1], 16384):
        acc += x[:, k:k + 16384].double() @ w[:, k:k + 16384].double().T
    y = acc.float() * (xs[:, None] * ws[None, :])
    return (y if bias is None else y + bias.float()).to(t)


def operands(m, n, k, seed, pad=0):
    g = rng(seed)
    x = torch.randint(-128, 128, (m, k + pad), generator=g, device="cuda", dtype=torch.int8)[:, :k]
    w = torch.randint(-128, 128, (n, k + pad), generator=g, device="cuda", dtype=torch.int8)[:, :k]
    return x, torch.rand(m, generator=g, device="cuda") + 0.01, w, torch.randn(n, generator=g, device="cuda")


SIZES = [(1, 1, 16), (1, 8, 128), (3, 129, 144), (8, 512, 1024), (16, 300, 1040), (17, 128, 2048), (31, 257, 528), (33, 1000, 2064),
         (64, 64, 4096), (65, 200, 512), (100, 640, 1152), (128, 128, 8192), (129, 384, 1024), (200, 1032, 3056),
         (256, 256, 256), (257, 513, 1168), (300, 2050, 640), (512, 1024, 4096), (777, 520, 2320), (1100, 1500, 1024),
         (40, 5120, 1024), (2, 8192, 512), (4, 100, 131056), (300, 100, 131056)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(far, m, n, k):
    x, xs, w, ws = operands(m, n, k, m + n + k)
    for i, t in enumerate(TYPES.values()):
        bias = None if (m + i) % 2 else torch.randn(n, generator=rng(5), device="cuda").to(t)
        y = far.gemm_int8(x, xs, w, ws, bias, out_dtype=t)
        assert torch.equal(y, product(x, xs, w, ws, bias, t)), (t, far.device_status())
    assert far.device_status() == 0


@pytest.mark.parametrize("m,n,k", [(5, 7, 1), (1, 3, 5), (70, 130, 100), (200, 65, 1001), (3, 300, 131071)])
def test_product_of_any_length(far, m, n, k):
    """k that TMA cannot step over, the longest k too."""
    x, xs, w, ws = operands(m, n, k, k)
    for t in TYPES.values():
        assert torch.equal(far.gemm_int8(x, xs, w, ws, out_dtype=t), product(x, xs, w, ws, None, t))


@pytest.mark.parametrize("m", [1, 16, 40, 130, 300])
@pytest.mark.parametrize("x0,w0", [(-128, -128), (127, -128), (127, 127), (-128, 127)])
def test_largest_sums(far, m, x0, w0):
    """Every product as large as it gets: sums of 2^24 a 1024 values, 2^31 - 2^14 at the longest; and large sums that a few small
    products follow or precede."""
    for k in (1024, 2048, 16384, 131056):
        x = torch.full((m, k), x0, dtype=torch.int8, device="cuda")
        w = torch.full((130, k), w0, dtype=torch.int8, device="cuda")
        w[1, k // 2:] = 1
        w[2, :k // 2] = -1
        w[3, ::2] = 0
        w[4, 1::2] = -w[4, 1::2].clamp(min=-127)
        w[5] = 0
        w[5, -1] = 1
        w[6, 1020:1024] = 3
        w[7, 1023] = 5
        one = torch.ones(m, device="cuda"), torch.ones(130, device="cuda")
        y = far.gemm_int8(x, one[0], w, one[1], out_dtype=torch.float32)
        assert torch.equal(y, product(x, one[0], w, one[1], None, torch.float32)), k


@pytest.mark.parametrize("m", [3, 90, 300])
def test_scales(far, m):
    """Zero, far, infinite and NaN scales: fl32(acc) times their product, or one after the other where that leaves binary32's
    normal numbers."""
    x, xs, w, ws = operands(m, 64, 512, 11)
    xs[0], ws[:6] = 0.0, torch.tensor([0.0, 1e30, 1e-30, float("inf"), float("nan"), 2.0 ** -149])
    xs[1], xs[2] = 1e30, 1e-30
    y = far.gemm_int8(x, xs, w, ws, out_dtype=torch.float32)
    acc = x.double() @ w.double().T
    want = (acc.float().double() * xs.double()[:, None] * ws.double()).float()
    fine = want.isfinite()
    assert bool((y[fine].double() - want[fine].double()).abs().le(2.0 ** -22 * want[fine].double().abs() + 2.0 ** -149).all())
    assert bool((y[~fine].isnan() | y[~fine].isinf()).all()) and bool((y[0, :3] == 0).all()) and bool(y[:, 4].isnan().all())


def test_empty(far):
    x, xs, w, ws = operands(4, 6, 32, 1)
    b = torch.arange(6.0, device="cuda")
    assert far.gemm_int8(x[:0], xs[:0], w, ws).shape == (0, 6)
    assert far.gemm_int8(x, xs, w[:0], ws[:0]).shape == (4, 0)
    y = far.gemm_int8(x[:, :0], xs, w[:, :0], ws, b, out_dtype=torch.float32)
    assert torch.equal(y, b.expand(4, 6))
    assert far.quant_rows_int8(torch.zeros(0, 8, device="cuda"))[0].shape == (0, 8)


@pytest.mark.parametrize("m,n,k", [(9, 200, 256), (70, 330, 512), (300, 330, 1024)])
@pytest.mark.parametrize("t", TYPES)
def test_strides_and_places(far, m, n, k, t):
    """Rows of wider matrices on either side, an output inside a larger one at every alignment, leading axes."""
    x, xs, w, ws = operands(m, n, k, 3, pad=48)
    want = product(x, xs, w, ws, None, TYPES[t])
    for left in (0, 1, 2, 8):
        big = torch.full((m + 2, n + 16), 5.0, device="cuda").to(TYPES[t])
        out = big[1:m + 1, left:left + n]
        assert far.gemm_int8(x, xs, w, ws, out_dtype=TYPES[t], out=out) is out
        assert torch.equal(out, want)
        big[1:m + 1, left:left + n] = 5.0
        assert bool((big == 5.0).all())
    xc = x.contiguous()
    y = far.gemm_int8(xc.view(1, m, k), xs.view(1, m), w, ws, out_dtype=TYPES[t])
    assert y.shape == (1, m, n) and torch.equal(y[0], want)
    odd = torch.empty(m * k + 3, dtype=torch.int8, device="cuda")[3:].view(m, k)  # off 16 bytes
    odd.copy_(x)
    assert torch.equal(far.gemm_int8(odd, xs, w, ws, out_dtype=TYPES[t]), want)


@pytest.mark.parametrize("m,n,k", [(4, 512, 1024), (60, 512, 1024), (300, 512, 2048)])
def test_streams_and_graphs(far, m, n, k):
    """A captured call replayed on new inputs, two graphs at once on two streams, explicit streams, a workspace given."""
    x, xs, w, ws = operands(m, n, k, 9)
    space = torch.empty(far.gemm_int8_workspace_bytes(m, n, k) + 16, dtype=torch.uint8, device="cuda")
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    far.gemm_int8(x, xs, w, ws, out=out, workspace=space)
    graphs, outs = [], []
    for _ in range(2):
        outs.append(torch.zeros_like(out))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            far.gemm_int8(x, xs, w, ws, out=outs[-1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for seed in (1, 2):
        x2, xs2, w2, ws2 = operands(m, n, k, seed)
        for a, b in ((x, x2), (xs, xs2), (w, w2), (ws, ws2)):
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
    if far.gemm_int8_workspace_bytes(m, n, k):
        with pytest.raises(far.FarError):
            far.gemm_int8(x, xs, w, ws, out=out, workspace=space[:16])
    assert far.device_status() == 0


def test_projection_behind_the_norm(far):
    """The run that the product is for: norm with int8 output, projection, its output quantised again, another projection."""
    g = rng(21)
    x, r = (torch.randn(50, 1024, generator=g, device="cuda").bfloat16() for _ in range(2))
    one = torch.ones(1024, device="cuda").bfloat16()
    w1 = (torch.randn(2048, 1024, generator=g, device="cuda") / 32).bfloat16()
    w2 = (torch.randn(1024, 2048, generator=g, device="cuda") / 45).bfloat16()
    (q1, s1), (q2, s2) = far.quant_rows_int8(w1), far.quant_rows_int8(w2)
    xq, xs, res = far.fused_add_rmsnorm_quant(x, r, one, 1e-6, "int8")
    out, res2 = far.fused_add_rmsnorm(x, r, one, 1e-6)
    oq, os = far.quant_rows_int8(out)
    assert torch.equal(xq, oq) and torch.equal(xs, os) and torch.equal(res, res2)  # the norm quantises as quant_rows_int8 does
    h = far.gemm_int8(xq, xs, q1, s1)
    assert torch.equal(h, product(xq, xs, q1, s1, None, torch.bfloat16))
    hq, hs = far.quant_rows_int8(h)
    y = far.gemm_int8(hq, hs, q2, s2, out_dtype=torch.float16)
    assert torch.equal(y, product(hq, hs, q2, s2, None, torch.float16))


def test_threads_on_their_own_streams(far):
    """Four threads, each with a stream, calling at once with the lock let go inside: every result its own."""
    import threading

    cases = [operands(m, 520, 1024, m) for m in (3, 70, 300, 700)]
    want = [product(*c, None, torch.bfloat16) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = [far.gemm_int8(*cases[i]) for _ in range(50)]
        s.synchronize()
        if not all(torch.equal(g, want[i]) for g in got):
            wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and far.device_status() == 0
