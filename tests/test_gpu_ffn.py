"""The gated feed-forward block on the GPU, against its formulas in 64 bits with derived bounds, and bit for bit where every
sum is exact; strides, places outputs must not touch, streams and graphs."""
import pytest
import torch

import ffn_ref as ref

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


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


def inputs(m, h, f, t, seed):
    g = rng(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return n(m, h).to(t), (2 * n(f, h) / h ** 0.5).to(t), (n(f, h) / h ** 0.5).to(t)


def integers(g, t, *shape, most=3):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(t)


# one token to several tiles of rows; few and many columns; hidden of one slice to many, with and without whole
# 16 bytes; ffn odd, so that outputs lie on every alignment
SIZES = [(1, 8, 8), (1, 256, 64), (1, 2056, 1000), (2, 64, 40), (7, 72, 136), (16, 512, 200), (17, 1024, 333), (32, 128, 64),
         (33, 1032, 264), (60, 520, 776), (64, 4096, 128), (65, 256, 129), (100, 2048, 300), (128, 136, 1024),
         (129, 512, 257), (200, 264, 512), (256, 256, 128), (257, 1024, 640), (300, 72, 2744), (777, 136, 1100), (1030, 320, 513),
         (40, 77, 50), (300, 5, 70), (5, 1, 3)]


@pytest.mark.parametrize("m,h,f", SIZES)
@pytest.mark.parametrize("t", TYPES)
def test_forward(far, t, m, h, f):
    name = ref.ACTS[(m + f) % 3]
    x, wg, wu = inputs(m, h, f, TYPES[t], m + h + f)
    want = ref.forward(x, wg, wu, name)
    got = far.gated_ffn(x, wg, wu, activation=name, save=True)
    for v, (w, e) in zip(got, want):
        assert v.shape == (m, f) and ref.within(v, w, e), far.device_status()
    assert torch.equal(far.gated_ffn(x, wg, wu, activation=name), got[0])
    assert far.device_status() == 0


@pytest.mark.parametrize("m,h,f", SIZES)
@pytest.mark.parametrize("t", TYPES)
def test_forward_exact_sums(far, t, m, h, f):
    """Small whole numbers: both projections are exact, so the kept ones are their roundings bit for bit."""
    g = rng(m * h + f)
    x, wg, wu = integers(g, TYPES[t], m, h), integers(g, TYPES[t], f, h), integers(g, TYPES[t], f, h)
    _, gate, up = far.gated_ffn(x, wg, wu, save=True)
    assert torch.equal(gate, (x.double() @ wg.double().T).float().to(TYPES[t]))
    assert torch.equal(up, (x.double() @ wu.double().T).float().to(TYPES[t]))


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("t", TYPES)
def test_activation_everywhere(far, t, name):
    """One value of hidden: gate and up are x itself, over every finite value of the type: out is act(x) x."""
    x = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32, device="cuda").to(torch.int16).view(TYPES[t])
    x = x[x.isfinite()][:, None]
    pad = torch.zeros(x.shape[0], 8, dtype=TYPES[t], device="cuda")
    pad[:, :1] = x
    one = torch.zeros(8, 8, dtype=TYPES[t], device="cuda")
    one[:, 0] = 1
    for m in (slice(0, 40), slice(None)):
        out = far.gated_ffn(pad[m], one, one, activation=name)
        v = x[m].double()
        want = ref.act(v, name) * v
        big = want.abs() > torch.finfo(TYPES[t]).max
        allowed = 2.0 ** -14 * want.abs() + ref.rounded(want.abs(), TYPES[t])
        ok = ((out.double() - want).abs() <= allowed) | (big & (out.isinf() | (out.double().abs() >= torch.finfo(TYPES[t]).max * 0.99)))
        assert bool(ok.all())


def test_non_finite(far):
    x = torch.zeros(4, 8, device="cuda").half()
    x[0, 0], x[1, 0], x[2, 0] = float("nan"), float("inf"), -float("inf")
    w = torch.zeros(8, 8, device="cuda").half()
    w[:, 0] = 1
    for name in ref.ACTS:
        out, gate, up = far.gated_ffn(x, w, w, activation=name, save=True)
        assert bool(out[0].isnan().all()) and bool((out[1] == float("inf")).all()) and bool(out[2].isnan().all())
        assert bool((out[3] == 0).all()) and bool((gate[1] == float("inf")).all())


@pytest.mark.parametrize("m,h,f", [(5, 72, 136), (300, 264, 200), (40, 77, 50)])
def test_nan_stays_in_its_row(far, m, h, f):
    """A NaN token, a NaN weight row: one row and one column of out are NaN, everything else is what it is without them (no kernel
    multiplies what lies past an edge); the same for dx and a NaN token of dout."""
    x, wg, wu = inputs(m, h, f, torch.bfloat16, 5)
    clean = far.gated_ffn(x, wg, wu)
    bad_x, bad_w = x.clone(), wu.clone()
    bad_x[m - 2], bad_w[f - 3, h - 1] = float("nan"), float("nan")
    out = far.gated_ffn(bad_x, wg, bad_w)
    bad = torch.zeros(m, f, dtype=torch.bool, device="cuda")
    bad[m - 2], bad[:, f - 3] = True, True
    assert torch.equal(out.isnan(), bad) and torch.equal(out[~bad], clean[~bad])
    args = gradients(m, h, f, torch.bfloat16, 6)
    clean = far.gated_ffn_backward(*args)
    dh = args[0].clone()
    dh[m - 2, f - 1] = float("nan")
    dx, dwg, dwu = far.gated_ffn_backward(dh, *args[1:])
    rows = torch.arange(m, device="cuda") == m - 2
    assert bool(dx[rows].isnan().all()) and torch.equal(dx[~rows], clean[0][~rows])
    for a, b in ((dwg, clean[1]), (dwu, clean[2])):
        assert bool(a[f - 1].isnan().all()) and torch.equal(a[:f - 1], b[:f - 1])


BACK = [(1, 8, 8), (1, 256, 64), (3, 64, 40), (16, 512, 200), (33, 1032, 333), (64, 128, 129), (65, 256, 1000), (100, 520, 264),
        (128, 136, 1024), (200, 264, 512), (257, 1024, 640), (333, 1032, 1100), (777, 136, 257), (1030, 320, 513), (40, 77, 50),
        (300, 5, 70)]


def gradients(m, h, f, t, seed):
    g = rng(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    return n(m, f), (1.5 * n(m, f)).to(t), n(m, f), n(m, h), (n(f, h) / h ** 0.5).to(t), (n(f, h) / h ** 0.5).to(t)


@pytest.mark.parametrize("m,h,f", BACK)
@pytest.mark.parametrize("t", TYPES)
def test_backward(far, t, m, h, f):
    name = ref.ACTS[(m + f) % 3]
    args = gradients(m, h, f, TYPES[t], m + h + f)
    got = far.gated_ffn_backward(*args, activation=name)
    for v, (w, e) in zip(got, ref.backward(*args, name)):
        assert v.shape == w.shape and ref.within(v, w, e), far.device_status()
    again = far.gated_ffn_backward(*args, activation=name)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert far.device_status() == 0


@pytest.mark.parametrize("m,h,f", BACK)
@pytest.mark.parametrize("t", TYPES)
def test_backward_exact_sums(far, t, m, h, f):
    """At gate = 32 every activation is its argument and its slope 1: with small whole numbers all sums are exact."""
    g = rng(m * h + f)
    t = TYPES[t]
    dh, up, x, wg, wu = (integers(g, t, *s, most=2) for s in ((m, f), (m, f), (m, h), (f, h), (f, h)))
    gate = torch.full((m, f), 32.0, device="cuda").to(t)
    for name in ref.ACTS:
        dx, dwg, dwu = far.gated_ffn_backward(dh, gate, up, x, wg, wu, activation=name)
        dg, du = (dh.double() * up.double()), 32 * dh.double()
        assert torch.equal(dx, (dg @ wg.double() + du @ wu.double()).float().to(t))
        assert torch.equal(dwg, (dg.T @ x.double()).float().to(t)) and torch.equal(dwu, (du.T @ x.double()).float().to(t))


@pytest.mark.parametrize("name", ref.ACTS)
def test_backward_against_differences(far, name):
    """The forward's own outputs differ along a direction as its gradients say.  With step d and loss L = sum(c out), out
    rounded to f16 by 2^-11 of itself (and binary32 sums): |L(+d) - L(-d)| / 2d is off by at most sum |c| 2^-11 |out| / d,
    and by d^2 / 6 of a third derivative, which is bounded by evaluating the reference's at d and 2 d; the gradients
    themselves by ref.backward's bounds along the direction."""
    x, wg, wu = inputs(24, 64, 40, torch.float16, 7)
    c = torch.randn(24, 40, generator=rng(8), device="cuda").half()
    _, gate, up = far.gated_ffn(x, wg, wu, activation=name, save=True)
    grads = far.gated_ffn_backward(c, gate, up, x, wg, wu, activation=name)
    bounds = ref.backward(c, gate, up, x, wg, wu, name)
    leaves = [x, wg, wu]
    d = 2.0 ** -4
    for i in range(3):
        v = integers(rng(30 + i), torch.float16, *leaves[i].shape, most=1) / 8
        moved = [[(w + s * d * v).half() if k == i else w for k, w in enumerate(leaves)] for s in (1, -1)]
        step = (moved[0][i].double() - moved[1][i].double())  # what was really added
        outs = [far.gated_ffn(*a, activation=name).double() for a in moved]
        found = float(((outs[0] - outs[1]) * c.double()).sum())
        exact = [ref.forward(*a, name)[0] for a in moved]
        want = float(((exact[0][0] - exact[1][0]) * c.double()).sum())
        allowed = float(sum((e * c.double().abs()).sum() for _, e in exact))
        assert abs(found - want) <= allowed
        along = float((grads[i].double() * step).sum())
        slack = float((bounds[i][1] * step.abs()).sum())
        # the exact difference against the exact derivative: the curvature's share, from 64-bit evaluations alone
        e64 = float((bounds[i][0] * step).sum())
        assert abs(along - found) <= allowed + slack + abs(want - e64)
        assert abs(want - e64) <= 0.05 * float((bounds[i][0] * step).abs().sum())


@pytest.mark.parametrize("h,f", [(64, 40), (0, 8), (64, 0)])
def test_empty(far, h, f):
    x, w = torch.zeros(0, h, device="cuda").half(), torch.ones(f, h, device="cuda").half()
    assert far.gated_ffn(x, w, w).shape == (0, f)
    d = torch.zeros(0, f, device="cuda").half()
    dx, dwg, dwu = far.gated_ffn_backward(d, d, d, x, w, w)
    assert dx.shape == (0, h) and bool((dwg == 0).all()) and bool((dwu == 0).all()) and dwg.shape == (f, h)
    x = torch.ones(3, h, device="cuda").half()
    out = far.gated_ffn(x, w, w)
    assert out.shape == (3, f) and (h > 0 or bool((out == 0).all()))
    d = torch.ones(3, f, device="cuda").half()
    dx, dwg, _ = far.gated_ffn_backward(d, d, d, x, w, w)
    assert dx.shape == (3, h) and (f > 0 or bool((dx == 0).all()))


@pytest.mark.parametrize("m,h,f", [(9, 256, 200), (70, 512, 136), (300, 520, 328)])
def test_strides_and_places(far, m, h, f):
    """Column slices of wider matrices on every side, outputs inside larger ones at several alignments, leading axes."""
    t = torch.bfloat16
    g = rng(5)
    wide = lambda r, c: torch.randn(r, c + 24, generator=g, device="cuda").to(t)[:, 8:c + 8] / 4  # noqa: E731
    x, wg, wu = wide(m, h), wide(f, h), wide(f, h)
    want = far.gated_ffn(x.contiguous(), wg.contiguous(), wu.contiguous(), save=True)
    for left in (0, 1, 2, 8):
        bigs = [torch.full((m + 2, f + 16), 5.0, device="cuda", dtype=t) for _ in range(3)]
        outs = [b[1:m + 1, left:left + f] for b in bigs]
        got = far.gated_ffn(x, wg, wu, save=True, out=outs[0], gate_out=outs[1], up_out=outs[2])
        for o, w, r, b in zip(outs, want, got, bigs):
            assert r is o and torch.equal(o, w)
            o.fill_(5.0)
            assert bool((b == 5.0).all())
    assert torch.equal(far.gated_ffn(x.contiguous().view(1, m, h), wg, wu)[0], want[0])
    odd = [torch.empty(v.numel() + 1, device="cuda", dtype=t)[1:].view(v.shape).copy_(v) for v in (x, wg, wu)]  # off 16 bytes
    for v, (w, e) in zip(far.gated_ffn(*odd, save=True), ref.forward(x, wg, wu, "silu")):
        assert ref.within(v, w, e)
    dh, gate, up = wide(m, f), wide(m, f), wide(m, f)
    want = far.gated_ffn_backward(*(v.contiguous() for v in (dh, gate, up, x, wg, wu)))
    for left in (0, 1, 8):
        bigs = [torch.full((r + 2, h + 16), 5.0, device="cuda", dtype=t) for r in (m, f, f)]
        outs = [b[1:-1, left:left + h] for b in bigs]
        got = far.gated_ffn_backward(dh, gate, up, x, wg, wu, dx=outs[0], dw_gate=outs[1], dw_up=outs[2])
        for o, w, r, b in zip(outs, want, got, bigs):
            assert r is o and torch.equal(o, w)
            o.fill_(5.0)
            assert bool((b == 5.0).all())


def test_leading_axes_and_one_weight_twice(far):
    """[batch, tokens, hidden] there and back, on a stream with every output and the workspace given; both weights one tensor."""
    t = torch.bfloat16
    x, w, _ = inputs(2 * 35, 264, 136, t, 3)
    dh = torch.randn(70, 136, generator=rng(4), device="cuda").to(t)
    flat = far.gated_ffn(x, w, w, save=True)
    back = far.gated_ffn_backward(dh, flat[1], flat[2], x, w, w)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.empty(2, 35, 136, device="cuda", dtype=t) for _ in range(3)]
    got = far.gated_ffn(x.view(2, 35, 264), w, w, save=True, out=outs[0], gate_out=outs[1], up_out=outs[2], stream=stream)
    grads = [torch.empty(2, 35, 264, device="cuda", dtype=t), torch.empty_like(w), torch.empty_like(w)]
    space = torch.empty(far.gated_ffn_backward_workspace_bytes(70, 136), dtype=torch.uint8, device="cuda")
    more = far.gated_ffn_backward(dh.view(2, 35, 136), got[1], got[2], x.view(2, 35, 264), w, w, dx=grads[0], dw_gate=grads[1],
                                  dw_up=grads[2], workspace=space, stream=stream)
    stream.synchronize()
    for a, b in zip((*got, *more), (*flat, *back)):
        assert torch.equal(a.view(b.shape), b)
    assert all(a is b for a, b in zip((*got, *more), (*outs, *grads)))
    for v, (e, allowed) in zip(flat, ref.forward(x, w, w, "silu")):
        assert ref.within(v, e, allowed)


@pytest.mark.parametrize("m,h,f", [(2, 512, 256), (50, 512, 256), (300, 512, 640)])
def test_streams_and_graphs(far, m, h, f):
    """Both ways captured and replayed on new inputs, two graphs at once on two streams, explicit streams, a workspace given."""
    t = torch.float16
    x, wg, wu = inputs(m, h, f, t, 1)
    dh = torch.randn(m, f, generator=rng(2), device="cuda").to(t)

    def both(stream=None, **kw):
        out, gate, up = far.gated_ffn(x, wg, wu, save=True, stream=stream)
        return out, *far.gated_ffn_backward(dh, gate, up, x, wg, wu, stream=stream, **kw)

    both()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(both())
    streams = [torch.cuda.Stream() for _ in range(2)]
    space = torch.empty(far.gated_ffn_backward_workspace_bytes(m, f), dtype=torch.uint8, device="cuda")
    for seed in (3, 4):
        for a, b in zip((x, wg, wu), inputs(m, h, f, t, seed)):
            a.copy_(b)
        want = both()
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for got in (*outs, *[both(s) for s in streams], both(workspace=space)):
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(far.FarError):
        both(workspace=space[:-16])
    assert far.device_status() == 0


def test_block_with_an_int8_way_out(far):
    """The run that these operators are for: norm, feed-forward block, its values quantised, the int8 projection back, the next
    norm with int8 output; each step against its definition on the step before."""
    g = rng(40)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, r = n(70, 512).bfloat16(), n(70, 512).bfloat16()
    one = torch.ones(512, device="cuda").bfloat16()
    wg, wu = (n(1400, 512) / 22).bfloat16(), (n(1400, 512) / 22).bfloat16()
    down = (n(512, 1400) / 37).bfloat16()
    dq, ds = far.quant_rows_int8(down)
    normed, res = far.fused_add_rmsnorm(x, r, one, 1e-6)
    h = far.gated_ffn(normed, wg, wu)
    w, e = ref.forward(normed, wg, wu, "silu")[0]
    assert ref.within(h, w, e)
    hq, hs = far.quant_rows_int8(h)
    y = far.gemm_int8(hq, hs, dq, ds)
    exact = (hq.double() @ dq.double().T) * (hs.double()[:, None] * ds.double())
    assert bool(((y.double() - exact).abs() <= (2.0 ** -22 + 2.0 ** -8) * exact.abs() + 2.0 ** -130).all())
    # (int8: half a code of either side, 2^-8 of a row's largest value, over 1400 products)
    true = h.double() @ down.double().T
    step = hs.double()[:, None] / 2 * down.double().abs().sum(1) + h.double().abs().sum(1)[:, None] * ds.double() / 2
    assert bool(((y.double() - true).abs() <= 1.01 * step + 2.0 ** -8 * true.abs() + 700 * hs.double()[:, None] * ds.double()).all())
    q, s, res2 = far.fused_add_rmsnorm_quant(y, res, one, 1e-6, "int8")
    out, res3 = far.fused_add_rmsnorm(y, res, one, 1e-6)
    oq, os_ = far.quant_rows_int8(out)
    assert torch.equal(q, oq) and torch.equal(s, os_) and torch.equal(res2, res3)
