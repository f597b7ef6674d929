"""The 128-block FP8 operators on the GPU: quantisation bit for bit against its definition (block_ref),
the norm's block-quantised output bit for bit against quantising the plain operation's output,
the product within the bound of its binary32 sums (block_ref.product), exactly where every sum
is exact; then a layer's run of them together."""
import numpy as np
import pytest
import torch

import far_gen
import oracle
from block_ref import BLOCK, nblocks, product, quantise, same_scales, same_values
from gpu_helpers import Guarded
from heads_ref import SMALLEST, half_step
from oracle_pins import bits_equal

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
PAIRS = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32"), ("f32", "f32"), ("f32", "bf16"), ("f32", "f16")]


@pytest.fixture(scope="module")
def far():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    far.set_launch_override()
    return far


def guarded_bytes(n):
    """A byte buffer between canary bands: (view, check)."""
    b = Guarded(((n + 3) // 4 + 1,), torch.float32)
    b.t.view(torch.int32).fill_(0x5A5A5A5A)
    v = b.t.view(torch.uint8)[:n]
    tail = b.t.view(torch.uint8)[n:]
    return v, lambda: b.guards_intact() and bool((tail == 0x5A).all())


# ---------------------------------------------------------------------------
# the norm's block-quantised output
# ---------------------------------------------------------------------------

def check_norm(far, d, where):
    x, r, w = d["x"].cuda(), d["r"].cuda(), d["w"].cuda()
    out, res = far.fused_add_rmsnorm(x, r, w, d["eps"])
    q, s, ro = far.fused_add_rmsnorm_quant_block(x, r, w, d["eps"])
    assert far.device_status() == 0
    assert q.dtype == E4M3 and torch.equal(ro.view(torch.uint8), res.view(torch.uint8)), f"{where}: residual_out"
    v, rs = quantise(out.cpu(), "row")
    assert same_scales(s, rs), f"{where}: scales"
    assert same_values(q, v), f"{where}: codes"
    out = far.rmsnorm(x, w, d["eps"])
    q, s = far.rmsnorm_quant_block(x, w, d["eps"])
    v, rs = quantise(out.cpu(), "row")
    assert same_scales(s, rs) and same_values(q, v), f"{where}: no residual"


@pytest.mark.parametrize("act,wd", PAIRS)
@pytest.mark.parametrize("hidden", [1, 8, 100, 128, 136, 1000, 2048, 4096, 5120, 8192])
def test_norm(far, act, wd, hidden):
    check_norm(far, far_gen.custom_inputs(act, wd, 33, hidden, seed=hidden, scale_lo=1e-3, scale_hi=30),
               f"{act}/{wd} {hidden}")


@pytest.mark.parametrize("tokens,hidden", [(1, 8192), (400, 5120), (700, 2560), (1500, 1024), (700, 6144), (330, 16384), (3, 65536)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_norm_plans(far, act, tokens, hidden):
    check_norm(far, far_gen.custom_inputs(act, act, tokens, hidden, seed=tokens, scale_lo=1e-2, scale_hi=50), f"{act} {tokens}x{hidden}")


def test_norm_schedules_and_plans(far):
    """Claimed rows (modes 0 and 2) and forced plans give the fixed stride's bits."""
    d = far_gen.custom_inputs("bf16", "bf16", 2500, 4096, seed=3)
    x, r, w = d["x"].cuda(), d["r"].cuda(), d["w"].cuda()
    want = far.fused_add_rmsnorm_quant_block(x, r, w, 1e-6) + far.rmsnorm_quant_block(x, w, 1e-6)
    same = lambda got: all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))  # noqa: E731
    run = lambda: far.fused_add_rmsnorm_quant_block(x, r, w, 1e-6) + far.rmsnorm_quant_block(x, w, 1e-6)  # noqa: E731
    try:
        for mode in (0, 2):
            far.set_row_schedule(mode)
            assert same(run()), f"schedule {mode}"
        far.set_row_schedule(1)
        for plan in [(1, 0, 0, 0), (0, 4, 1, 2), (0, 8, 1, 0), (0, 2, 0, 0)]:
            far.set_launch_override(*plan)
            assert same(run()), f"plan {plan}"
    finally:
        far.set_row_schedule(1)
        far.set_launch_override()


def test_norm_against_the_oracle(far):
    """The oracle's out quantised: residual_out and, wherever out agrees over a block, the block bit for bit."""
    d = far_gen.custom_inputs("bf16", "bf16", 64, 2048, seed=4)
    q, s, ro = far.fused_add_rmsnorm_quant_block(d["x"].cuda(), d["r"].cuda(), d["w"].cuda(), d["eps"])
    out, res = oracle.fused_add_rmsnorm(d["x"], d["r"], d["w"], d["eps"], d["act"], d["wd"])
    assert bits_equal(ro.cpu(), res)
    v, rs = quantise(out, "row")
    same = s.cpu() == rs
    assert float(same.float().mean()) > 0.99
    codes = q.float().double().cpu().view(64, -1, BLOCK)[same] == v.view(64, -1, BLOCK)[same]
    assert float(codes.float().mean()) > 0.99  # out may be an ulp off in under 1 % of the elements


def test_norm_strides_in_place_and_special_rows(far):
    d = far_gen.custom_inputs("f16", "f16", 40, 1024, seed=2)
    x, r, w = d["x"].cuda(), d["r"].cuda(), d["w"].cuda()
    x[3] = 0.0
    r[3] = 0.0
    x[4, 7] = float("nan")
    x[5, 900] = float("inf")
    wide = torch.zeros(40, 2048, dtype=torch.float16, device="cuda")[:, 8:1032]
    wide.copy_(x)
    want = far.fused_add_rmsnorm_quant_block(x, r, w, 1e-6)
    r2 = r.clone()
    got = far.fused_add_rmsnorm_quant_block(wide, r2, w, 1e-6, residual_out=r2)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    out, _ = far.fused_add_rmsnorm(x, r, w, 1e-6)
    v, rs = quantise(out.cpu(), "row")
    assert same_scales(want[1], rs) and same_values(want[0], v)
    assert (want[1][3] == 0).all() and want[1][4].isnan().any()
    q3 = far.rmsnorm_quant_block(x.view(4, 10, 1024), w, 1e-6)
    assert q3[0].shape == (4, 10, 1024) and q3[1].shape == (4, 10, 8)


@pytest.mark.parametrize("kind", [0, 1])
def test_quantised_outputs_in_place(far, kind):
    """residual_out written over x or over the residual gives the same bits as into a buffer of its own, on
    the staged and on the generic kernel (which reads the rows again after the first sweep)."""
    d = far_gen.custom_inputs("bf16", "bf16", 30, 1024, seed=7)
    x, r, w = d["x"].cuda(), d["r"].cuda(), d["w"].cuda()
    try:
        far.set_launch_override(kind)
        for call in (lambda a, b, o: far.fused_add_rmsnorm_quant(a, b, w, 1e-6, "int8", residual_out=o),
                     lambda a, b, o: far.fused_add_rmsnorm_quant(a, b, w, 1e-6, "fp8", residual_out=o),
                     lambda a, b, o: far.fused_add_rmsnorm_quant_block(a, b, w, 1e-6, residual_out=o)):
            want = call(x, r, None)
            for over in (0, 1):
                a, b = x.clone(), r.clone()
                got = call(a, b, (a, b)[over])
                assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got, want))
    finally:
        far.set_launch_override()


# ---------------------------------------------------------------------------
# quantising a matrix
# ---------------------------------------------------------------------------

def check_quant(far, x, block, transpose, where):
    r, c = (x.shape[1], x.shape[0]) if transpose else tuple(x.shape)
    q, intact = guarded_bytes(r * c)
    s = Guarded((r if block == "row" else nblocks(r), nblocks(c)), torch.float32)
    far.quant_block_fp8(x, block, transpose, q=q.view(r, c), scale=s.t)
    assert far.device_status() == 0
    assert intact() and s.guards_intact(), f"{where}: a store landed outside its output"
    v, rs = quantise(x.cpu().T if transpose else x.cpu(), block)
    assert same_scales(s.t, rs), f"{where}: scales"
    assert same_values(q.view(r, c), v), f"{where}: codes"


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("act", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", [(1, 1), (1, 8192), (3, 64), (128, 128), (129, 136), (250, 1000), (131, 77), (16, 4096), (400, 257),
                                  (1000, 512), (5, 12345)], ids=str)
def test_quant(far, size, act, block, transpose):
    g = torch.Generator(device="cuda").manual_seed(sum(size))
    x = torch.randn(size, generator=g, device="cuda") * torch.exp(2 * torch.randn(size[0], 1, generator=g, device="cuda"))
    check_quant(far, x.to(TYPES[act]), block, transpose, f"{size} {act} {block} {transpose}")


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_quant_values(far, act, block, transpose):
    """Every 16-bit magnitude in some block: subnormals, the tiny-block bound, NaN, infinities, zero blocks."""
    t = TYPES[act]
    x = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16).view(512, 128).to(t)
    check_quant(far, x, block, transpose, "all bf16")
    y = torch.randn(256, 256, device="cuda")
    y[:128, :128] *= 2.0 ** -101
    y[128:, :128] = 0.0
    y[130, 200] = float("nan")
    y[5, 140] = float("-inf")
    check_quant(far, y.to(t), block, transpose, "special")


def test_quant_strides(far):
    x = torch.randn(300, 1024, device="cuda").bfloat16()
    for view in (x[:, 128:640], x[:, 3:300], x[::2], x[7:9, :33]):
        for block in ("row", "tile"):
            for tr in (False, True):
                check_quant(far, view, block, tr, f"{view.shape} {view.stride()}")
    with pytest.raises(ValueError, match="contiguous"):
        far.quant_block_fp8(x.T)
    q, s = far.quant_block_fp8(torch.empty(0, 128, device="cuda"))
    assert q.shape == (0, 128) and s.shape == (0, 1)


def test_far_rows(far):
    """Rows past 2^32 bytes, in and out."""
    x = torch.empty(3, (1 << 31) + 16, dtype=torch.bfloat16, device="cuda")[:, :256]
    x.copy_(torch.randn(3, 256, device="cuda"))
    check_quant(far, x, "row", False, "far rows")
    check_quant(far, x, "tile", True, "far rows")
    n = 40000
    big = torch.randn(1, 128, device="cuda").bfloat16().expand(n, 128).contiguous().repeat(1, 1024)  # 40000 x 131072
    q, s = far.quant_block_fp8(big, "tile")
    v, rs = quantise(big[:128, :128].cpu(), "tile")
    assert same_values(q[-64:, -128:], v[:64]) and bool((s == rs.cuda()).all())
    del q, s
    qt, st = far.quant_block_fp8(big, "row", transpose=True)
    assert bool((st == st[:128].repeat(1024, 1)).all()) and torch.equal(qt[-128:].view(torch.uint8), qt[:128].view(torch.uint8))


# ---------------------------------------------------------------------------
# the product
# ---------------------------------------------------------------------------

def operands(m, n, k, rows, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    code = lambda r: torch.randint(0, 256, (r, k), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)  # noqa: E731
    clean = lambda c: torch.where((c & 0x7F) == 0x7F, torch.zeros_like(c), c)  # NaN codes apart  # noqa: E731
    scale = lambda r: torch.exp(torch.randn(r, nblocks(k), generator=g, device="cuda"))  # noqa: E731
    return clean(code(m)), scale(m), clean(code(n)), scale(n if rows == "row" else nblocks(n))


def check_gemm(far, xq, xs, wq, ws, dtype, where, out=None):
    m, n = xq.shape[0], wq.shape[0]
    o = Guarded((m, n), dtype) if out is None else None
    y = far.gemm_fp8_block(xq, xs, wq, ws, out_dtype=dtype, out=o.t if o else out)
    assert far.device_status() == 0
    assert o is None or o.guards_intact(), f"{where}: a store landed outside its output"
    ref, err = product(xq, xs, wq, ws)
    top = torch.finfo(dtype).max
    fine = (ref.abs() + err) * (1 + half_step(dtype)) < top  # fp16: past the range the result is infinite
    allowed = err + half_step(dtype) * (ref.abs() + err) + SMALLEST[dtype]
    off = (y.double() - ref).abs()
    bad = fine & ~(off <= allowed)
    assert not bad.any(), f"{where}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / allowed)[fine].max()):.3g}"
    over = (ref.abs() - err) > top * (1 + half_step(dtype) * 2)
    assert bool((y[over].isinf()).all())
    return y


GEMM = [(1, 1, 16), (1, 8, 128), (1, 130, 256), (2, 128, 144), (3, 300, 1040), (7, 256, 512), (16, 384, 2048), (17, 1000, 640),
        (33, 129, 128), (64, 512, 1024), (65, 257, 272), (100, 640, 384), (128, 128, 128), (129, 385, 528), (200, 2056, 512),
        (256, 512, 4096), (300, 300, 304), (513, 768, 256), (1000, 1544, 784), (2048, 2048, 512),
        (600, 777, 640), (3000, 1102, 256), (1025, 2049, 128), (3000, 520, 2064)]


@pytest.mark.parametrize("rows", ["tile", "row"])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("size", GEMM, ids=str)
def test_gemm(far, size, dtype, rows):
    check_gemm(far, *operands(*size, rows, seed=sum(size)), TYPES[dtype], f"{size} {dtype} {rows}")


@pytest.mark.parametrize("rows", ["tile", "row"])
@pytest.mark.parametrize("size", [(1, 5, 1), (3, 130, 127), (70, 65, 129), (130, 200, 333), (64, 64, 1000)], ids=str)
def test_gemm_any_k(far, size, rows):
    """k that TMA cannot step over: the plain kernel."""
    check_gemm(far, *operands(*size, rows), torch.float32, f"{size} {rows}")


@pytest.mark.parametrize("rows", ["tile", "row"])
@pytest.mark.parametrize("size", [(1, 128, 1024), (5, 300, 2064), (48, 256, 8192), (150, 400, 1040), (700, 1100, 2000), (1024, 1024, 4096)],
                         ids=str)
def test_gemm_exact(far, size, rows):
    """Small integers and scales that are powers of two: every partial sum is exact in binary32 in any
    order (|x w| <= 16, at most 2^13 of them, scales within 2^2 of one another), so are the results."""
    m, n, k = size
    g = torch.Generator(device="cuda").manual_seed(k)
    ints = lambda r: torch.randint(-4, 5, (r, k), generator=g, device="cuda").float().to(E4M3)  # noqa: E731
    pows = lambda r: torch.exp2(torch.randint(-1, 2, (r, nblocks(k)), generator=g, device="cuda").float())  # noqa: E731
    x, xs, w, ws = ints(m), pows(m), ints(n), pows(n if rows == "row" else nblocks(n))
    y = far.gemm_fp8_block(x, xs, w, ws, out_dtype=torch.float32)
    ref, _ = product(x, xs, w, ws)
    assert torch.equal(y.double(), ref)


def test_gemm_layouts(far):
    """Row strides of both operands and the output, three axes, float8 views, misaligned operands."""
    m, n, k = 70, 200, 384
    xq, xs, wq, ws = operands(m, n, k, "tile")
    want = far.gemm_fp8_block(xq, xs, wq, ws)
    wide_x, wide_w = torch.zeros(m, 640, dtype=torch.uint8, device="cuda"), torch.zeros(n, 400, dtype=torch.uint8, device="cuda")
    vx, vw = wide_x[:, 16:16 + k], wide_w[:, :k]
    vx.copy_(xq)
    vw.copy_(wq)
    out = torch.full((m, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    got = far.gemm_fp8_block(vx, xs, vw, ws, out=out[:, 8:8 + n])
    assert torch.equal(got, want)
    assert (out[:, :8] == 7).all() and (out[:, 8 + n:] == 7).all()
    assert torch.equal(far.gemm_fp8_block(xq.view(E4M3).view(7, 10, k), xs.view(7, 10, -1), wq.view(E4M3), ws).view(m, n), want)
    for off in (1, 8):  # off a 16-byte boundary: the plain kernel, within the same bound
        buf = torch.empty(m * k + off, dtype=torch.uint8, device="cuda")[off:].view(m, k)
        buf.copy_(xq)
        check_gemm(far, buf, xs, wq, ws, torch.float32, "misaligned x")
    odd = torch.empty(m, n + 1, dtype=torch.bfloat16, device="cuda")[:, 1:]
    assert torch.equal(far.gemm_fp8_block(xq, xs, wq, ws, out=odd), want)


@pytest.mark.parametrize("m", [3, 200, 700])
def test_gemm_special_values(far, m):
    """NaN codes stay in their row or column; zero scales give zeros, also beside a large block; infinite scales."""
    n, k = 384, 512
    xq, xs, wq, ws = operands(m, n, k, "row")
    xq[1, 5] = 0x7F
    wq[300, 130] = 0xFF
    xs[2] = 0.0
    ws[10] = 0.0
    y = far.gemm_fp8_block(xq, xs, wq, ws, out_dtype=torch.float32)
    nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    nan[1], nan[:, 300] = True, True
    assert bool((y.isnan() == nan).all())
    assert (y[2][~nan[2]] == 0).all() and (y[:, 10][~nan[:, 10]] == 0).all()


def test_gemm_empty(far):
    e = torch.empty(0, 256, dtype=torch.uint8, device="cuda")
    xq, xs, wq, ws = operands(4, 128, 256, "tile")
    assert far.gemm_fp8_block(e, xs[:0], wq, ws).shape == (0, 128)
    y = far.gemm_fp8_block(xq[:, :0], xs[:, :0], wq[:, :0], ws[:, :0], out=torch.full((4, 128), 3.0, device="cuda", dtype=torch.bfloat16))
    assert (y == 0).all()


def test_gemm_same_bits_every_run(far):
    for m in (4, 100, 600):
        a = operands(m, 1024, 2048, "tile")
        first = far.gemm_fp8_block(*a)
        for _ in range(5):
            assert torch.equal(far.gemm_fp8_block(*a), first)


def test_plain_launches_give_the_same_bits(far):
    """With programmatic dependent launch off (far_set_programmatic_launch), a run of dependent calls is the same."""
    x, r = torch.randn(40, 1024, device="cuda").bfloat16(), torch.randn(40, 1024, device="cuda").bfloat16()
    w, nw = torch.randn(768, 1024, device="cuda").bfloat16(), torch.ones(1024, device="cuda").bfloat16()
    table, pos, one = far.rope_table(64, 128), torch.arange(40, device="cuda"), torch.ones(128, device="cuda").bfloat16()

    def run():
        wq, ws = far.quant_block_fp8(w, block="tile")
        xq, xs, res = far.fused_add_rmsnorm_quant_block(x, r, nw, 1e-6)
        qkv = far.gemm_fp8_block(xq, xs, wq, ws).view(40, 6, 128)
        y = far.qk_norm_rope(qkv[:, :4], qkv[:, 4:], one, one, 1e-6, table, pos)
        return (res, qkv, *y, *far.qk_norm_rope_backward(*y, qkv[:, :4], qkv[:, 4:], one, one, 1e-6, table, pos))

    want = [run() for _ in range(3)]
    try:
        far.set_programmatic_launch(False)
        got = run()
    finally:
        far.set_programmatic_launch(True)
    for other in want[1:] + [got]:
        assert all(torch.equal(a, b) for a, b in zip(other, want[0]))


def test_gemm_streams_and_graphs(far):
    """Calls on three streams at once, and two captured graphs replayed on new values."""
    sets = [operands(m, 1024, 1024, "tile", seed=m) for m in (3, 130, 512)]
    want = [far.gemm_fp8_block(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[far.gemm_fp8_block(*a, stream=st) for a in sets] for st in streams for _ in range(4)]
    for st in streams:
        torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(y, w) for g in got for y, w in zip(g, want))
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append([far.gemm_fp8_block(*a) for a in sets])
    for a in sets:
        a[1].mul_(2.0)
    for g in graphs:
        g.replay()
    want = [far.gemm_fp8_block(*a) for a in sets]
    assert all(torch.equal(y, w) for o in outs for y, w in zip(o, want))


# ---------------------------------------------------------------------------
# a layer's run of them
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_attention_inputs_of_a_layer(far, tokens):
    """norm -> FP8 projection -> per-head norm and rotation in place, against the same steps in 64 bits
    from the codes on; then the way back: the heads' gradients, dx and dw by the block products."""
    from heads_ref import backward, forward, within

    hidden, h, hk, d = 1024, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(tokens)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, r = n(tokens, hidden).bfloat16(), n(tokens, hidden).bfloat16()
    nw, qw, kw = (1 + 0.1 * n(hidden)).bfloat16(), (1 + 0.1 * n(d)).bfloat16(), (1 + 0.1 * n(d)).bfloat16()
    weight = (n((h + 2 * hk) * d, hidden) / 32).bfloat16()
    table = far.rope_table(4096, d, base=1e6)
    pos = torch.arange(tokens, device="cuda") + 1000
    wq, ws = far.quant_block_fp8(weight, block="tile")
    xq, xs, res = far.fused_add_rmsnorm_quant_block(x, r, nw, 1e-6)
    qkv = far.gemm_fp8_block(xq, xs, wq, ws)
    ref, err = product(xq, xs, wq, ws)
    within(qkv, ref, err, "projection")
    heads = qkv.clone().view(tokens, h + 2 * hk, d)
    q, k = heads[:, :h], heads[:, h:h + hk]
    far.qk_norm_rope(q, k, qw, kw, 1e-6, table, pos, q_out=q, k_out=k)
    orig = qkv.view(tokens, h + 2 * hk, d)
    within(q, *forward(orig[:, :h], qw, 1e-6, table, pos, "half"), "queries")
    within(k, *forward(orig[:, h:h + hk], kw, 1e-6, table, pos, "half"), "keys")
    assert torch.equal(heads[:, h + hk:], orig[:, h + hk:])
    dy = n(tokens, h + 2 * hk, d).bfloat16()
    dq, dk, dqw, dkw = far.qk_norm_rope_backward(dy[:, :h], dy[:, h:h + hk], orig[:, :h], orig[:, h:h + hk], qw, kw, 1e-6, table,
                                                 pos)
    rdx, ex, rdw, ew = backward(dy[:, :h], orig[:, :h], qw, 1e-6, table, pos, "half")
    within(dq, rdx, ex, "dq")
    within(dqw, rdw, ew, "dq_weight")
    grad = torch.cat([dq, dk, dy[:, h + hk:]], 1).reshape(tokens, -1)
    normed, _ = far.fused_add_rmsnorm(x, r, nw, 1e-6)
    a, b = far.quant_block_fp8(grad), far.quant_block_fp8(weight, block="tile", transpose=True)
    check_gemm(far, *a, *b, torch.bfloat16, "dx")
    a, b = far.quant_block_fp8(grad, transpose=True), far.quant_block_fp8(normed, transpose=True)
    dw = check_gemm(far, *a, *b, torch.float32, "dw")
    # and what eight bits cost: each factor within 2^-4 of itself (half an E4M3 step, plus blocks'
    # smallest values), so a product within 2^-3 of its magnitude
    full = grad.double().T @ normed.double()
    size = grad.double().abs().T @ normed.double().abs()
    assert bool(((dw.double() - full).abs() <= 0.13 * size + 1e-2 * size.mean()).all())
    assert dw.shape == weight.shape
    assert np.isfinite(float(dw.sum()))


def test_quant_more_tile_rows_than_one_grid_axis(far):
    """More than 32768 rows of tiles (blockIdx.z takes part): each tile's values depend on its own rows alone, so those
    behind the first 32768 equal quantising them apart, which the definition checks."""
    behind = 32768 * BLOCK
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(behind + 32768 + 200, 8, generator=g, device="cuda").half()
    for block in ("row", "tile"):
        for transpose in (False, True):
            q, s = far.quant_block_fp8(x, block, transpose)
            assert far.device_status() == 0
            for cut in (slice(0, 384), slice(behind - 256, behind + 384), slice(behind + 32768 - 128, None)):
                part = x[cut]
                v, rs = quantise(part.cpu().T if transpose else part.cpu(), block)
                lo = cut.start // BLOCK
                if transpose:
                    got, sc = q[:, cut], s[:, lo:lo + nblocks(part.shape[0])]
                elif block == "tile":
                    got, sc = q[cut], s[lo:lo + nblocks(part.shape[0])]
                else:
                    got, sc = q[cut], s[cut]
                assert same_scales(sc, rs) and same_values(got.contiguous(), v), f"{block} {transpose} {cut}"
