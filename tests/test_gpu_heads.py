"""The per-head norm and rotation and their gradients on the GPU against the definition in 64
bits (tolerances: heads_ref), at the sizes, layouts and positions where they can go wrong."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import Guarded
from heads_ref import backward, forward, rows_of, within

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def far():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    return far


def make(tokens, h, hk, d, rot, act, wd=None, seed=0, rows=4096):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, wt = TYPES[act], TYPES[wd or act]
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = {"q": (n(tokens, h, d) * torch.exp(n(tokens, h, 1))).to(t), "k": (n(tokens, hk, d) * 3).to(t) if hk else None,
         "qw": (1 + 0.2 * n(d)).to(wt), "kw": (1 + 0.2 * n(d)).to(wt) if hk else None, "eps": 1e-6,
         "dq": n(tokens, h, d).to(t), "dk": n(tokens, hk, d).to(t) if hk else None}
    s["pos"] = torch.randint(0, rows, (tokens,), generator=g, device="cuda")
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f
    s["table"] = torch.cat([a.cos(), a.sin()], 1).float().contiguous()
    return s


def guarded(x):
    return None if x is None else Guarded(tuple(x.shape), x.dtype)


def check_forward(far, s, pairs, where, norm=True):
    inter = pairs == "inter"
    out = [guarded(s["q"]), guarded(s["k"])]
    o = [x and x.t for x in out]
    if norm:
        got = far.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"], s["pos"], interleaved=inter,
                               q_out=o[0], k_out=o[1])
    else:
        got = far.rope(s["q"], s["k"], s["table"], s["pos"], interleaved=inter, q_out=o[0], k_out=o[1])
    assert far.device_status() == 0
    for x, w, y, b in ((s["q"], s["qw"], got[0], out[0]), (s["k"], s["kw"], got[1], out[1])):
        if x is None:
            assert y is None
            continue
        ref, err = forward(x, w if norm else None, s["eps"], s["table"], s["pos"], pairs)
        within(y, ref, err, f"{where} norm={norm}")
        assert b.guards_intact(), f"{where}: a store landed outside its output"


def check_backward(far, s, pairs, where):
    out = [guarded(s["q"]), guarded(s["k"])]
    got = far.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"], s["pos"],
                                    interleaved=pairs == "inter", dq=out[0].t, dk=out[1] and out[1].t)
    assert far.device_status() == 0
    for x, dy, w, dx, dw, b in ((s["q"], s["dq"], s["qw"], got[0], got[2], out[0]),
                                (s["k"], s["dk"], s["kw"], got[1], got[3], out[1])):
        if x is None:
            assert dx is None and dw is None
            continue
        rdx, ex, rdw, ew = backward(dy, x, w, s["eps"], s["table"], s["pos"], pairs)
        within(dx, rdx, ex, f"{where} dx")
        assert dw.dtype == torch.float32
        within(dw, rdw, ew, f"{where} dw")
        assert b.guards_intact(), f"{where}: a store landed outside its output"


# tokens, query heads, key heads, head_dim, rot_dim: the vector kernels' lane counts (1 .. 32), odd
# chunk counts, parts of a head; then heads that only the scalar kernels take
SIZES = [(1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (3, 5, 0, 128, 128), (7, 4, 2, 96, 96), (33, 8, 2, 80, 32),
         (17, 3, 3, 128, 64), (5, 2, 2, 256, 256), (9, 2, 1, 512, 512), (6, 3, 1, 16, 16), (11, 2, 2, 72, 32),
         (600, 32, 8, 128, 128), (2, 130, 1, 64, 64), (70, 7, 1, 192, 48),
         (5, 2, 1, 66, 66), (4, 3, 2, 100, 50), (2, 2, 2, 2, 2), (3, 1, 1, 2048, 1024), (5, 2, 1, 63, 62),
         (260, 3, 2, 90, 20)]


@pytest.mark.parametrize("pairs", ["half", "inter"])
@pytest.mark.parametrize("act", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(far, size, act, pairs):
    s = make(*size, act, seed=size[0] + size[3])
    check_forward(far, s, pairs, f"{size} {act} {pairs}")
    check_forward(far, s, pairs, f"{size} {act} {pairs}", norm=False)


@pytest.mark.parametrize("pairs", ["half", "inter"])
@pytest.mark.parametrize("act", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(far, size, act, pairs):
    check_backward(far, make(*size, act, seed=size[0] + size[3] + 1), pairs, f"{size} {act} {pairs}")


@pytest.mark.parametrize("act,wd", [("bf16", "f32"), ("f16", "f32"), ("f32", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("size", [(9, 4, 2, 128, 128), (5, 2, 1, 66, 66)], ids=str)
def test_weight_types(far, size, act, wd):
    s = make(*size, act, wd)
    check_forward(far, s, "half", f"{size} {act}/{wd}")
    check_backward(far, s, "half", f"{size} {act}/{wd}")


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_rope_backward_is_the_transpose(far, act):
    """<rope(x), y> = <x, rope_backward(y)>, and the value itself, with a scaled table."""
    s = make(40, 4, 2, 128, 96, act)
    s["table"] *= 1.25
    dq, dk = far.rope_backward(s["dq"], s["dk"], s["table"], s["pos"])
    for y, d in ((s["dq"], dq), (s["dk"], dk)):
        c, sn = rows_of(s["table"], s["pos"])
        ref, err = forward(y, None, 0.0, torch.cat([c, -sn], -1)[:, 0], torch.arange(40, device="cuda"), "half")
        within(d, ref, err, "rope_backward")


def test_gradients_against_differences(far):
    """Central differences of the definition in 64 bits along random directions: with h = 1e-4
    they are within 1e-6 of the derivative here (h^2 times a third derivative of order one,
    and 1e-16 / h), far below the kernels' own allowance."""
    s = make(6, 3, 2, 64, 64, "f32", seed=3)
    dq, dk, dqw, dkw = far.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"],
                                                 s["pos"])
    g = torch.Generator(device="cuda").manual_seed(8)
    for x, w, dy, dx, dw in ((s["q"], s["qw"], s["dq"], dq, dqw), (s["k"], s["kw"], s["dk"], dk, dkw)):
        _, ex, _, ew = backward(dy, x, w, s["eps"], s["table"], s["pos"], "half")
        for _ in range(4):
            v = torch.randn(x.shape, generator=g, device="cuda").double()
            vw = torch.randn(w.shape, generator=g, device="cuda").double()

            def loss(h):
                y, _ = forward64(x.double() + h * v, w.double() + h * vw, s)
                return (y * dy.double()).sum()

            def forward64(a, b, s):
                return forward(a, b, s["eps"], s["table"], s["pos"], "half")

            h = 1e-4
            diff = float((loss(h) - loss(-h)) / (2 * h))
            dot = float((dx.double() * v).sum() + (dw.double() * vw).sum())
            allowed = float(((ex + 2.0 ** -24 * dx.abs()) * v.abs()).sum() + ((ew + 2.0 ** -24 * dw.abs()) * vw.abs()).sum())
            assert abs(diff - dot) <= allowed + 1e-5 * (1 + abs(diff)), (diff, dot)


# ---------------------------------------------------------------------------
# layouts
# ---------------------------------------------------------------------------

def test_packed_projection_in_place(far):
    """q and k as views of a packed [tokens, (h + 2 hk) d] projection, in place; the values untouched."""
    for act, d in (("bf16", 128), ("f32", 96), ("f16", 66)):
        s = make(37, 6, 2, d, d // 2 * 2, act)
        v = torch.randn(37, 2, d, device="cuda").to(TYPES[act])
        qkv = torch.cat([s["q"], s["k"], v], 1).reshape(37, -1).contiguous()
        q, k = qkv.view(37, 10, d)[:, :6], qkv.view(37, 10, d)[:, 6:8]
        a, b = far.qk_norm_rope(q, k, s["qw"], s["kw"], s["eps"], s["table"], s["pos"], q_out=q, k_out=k)
        assert a.data_ptr() == qkv.data_ptr()
        for x, w, y in ((s["q"], s["qw"], q), (s["k"], s["kw"], k)):
            within(y, *forward(x, w, s["eps"], s["table"], s["pos"], "half"), f"packed {act} {d}")
        assert torch.equal(qkv.view(37, 10, d)[:, 8:], v)


def test_interleaved_projection_in_place(far):
    """q, k and v interleaved head by head, [tokens, heads, 3, d]: in place, values untouched; one token too."""
    for tokens in (19, 1):
        s = make(tokens, 4, 4, 64, 64, "bf16")
        v = torch.randn(tokens, 4, 64, device="cuda").bfloat16()
        buf = torch.stack([s["q"], s["k"], v], 2).contiguous()
        q, k = buf[:, :, 0], buf[:, :, 1]
        far.qk_norm_rope(q, k, s["qw"], s["kw"], s["eps"], s["table"], s["pos"], q_out=q, k_out=k)
        assert far.device_status() == 0
        for x, w, y in ((s["q"], s["qw"], q), (s["k"], s["kw"], k)):
            within(y, *forward(x, w, s["eps"], s["table"], s["pos"], "half"), f"interleaved {tokens}")
        assert torch.equal(buf[:, :, 2], v)


def test_layouts_give_the_same_bits(far):
    """Head-major buffers, token strides with gaps, four axes, int32 positions: the contiguous call's bits."""
    s = make(24, 4, 2, 128, 128, "bf16")
    args = (s["qw"], s["kw"], s["eps"], s["table"])
    want = far.qk_norm_rope(s["q"], s["k"], *args, s["pos"])
    major = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (s["q"], s["k"])]
    out = [torch.empty_like(m) for m in major]
    assert out[0].stride() == major[0].stride()
    got = far.qk_norm_rope(*major, *args, s["pos"], q_out=out[0], k_out=out[1])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    wide = torch.zeros(24, 9, 4, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 3] = s["q"]
    got = far.qk_norm_rope(wide[:, 3], s["k"], *args, s["pos"].int())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = far.qk_norm_rope(s["q"].view(2, 12, 4, 128), s["k"].view(2, 12, 2, 128), *args, s["pos"].view(2, 12))
    assert all(torch.equal(a.reshape(24, -1, 128), b) for a, b in zip(got, want))
    with pytest.raises(ValueError, match="collapse"):
        far.rope(s["q"].view(2, 12, 4, 128).transpose(0, 1), None, s["table"], s["pos"])


def test_broadcast_inputs(far):
    """One key head read by all (head stride 0), one token's gradient for all (token stride 0)."""
    s = make(10, 4, 2, 64, 64, "bf16")
    one = s["k"][:, :1].expand(10, 3, 64)
    y, _ = far.qk_norm_rope(one, None, s["qw"], None, s["eps"], s["table"], s["pos"])
    within(y, *forward(one, s["qw"], s["eps"], s["table"], s["pos"], "half"), "broadcast head")
    dy = s["dq"][:1].expand(10, 4, 64)
    dx, _, dw, _ = far.qk_norm_rope_backward(dy, None, s["q"], None, s["qw"], None, s["eps"], s["table"], s["pos"])
    rdx, ex, rdw, ew = backward(dy, s["q"], s["qw"], s["eps"], s["table"], s["pos"], "half")
    within(dx, rdx, ex, "broadcast dy")
    within(dw, rdw, ew, "broadcast dy")
    with pytest.raises(far.FarError):
        far.rope(one, None, s["table"], s["pos"], q_out=one)  # an output in one place


def test_misaligned_buffers(far):
    """Buffers an element off a 16-byte boundary, and a table 4 bytes off, take the scalar kernels."""
    s = make(9, 3, 2, 128, 128, "bf16")
    for name in ("q", "k", "dq", "dk"):
        buf = torch.empty(s[name].numel() + 1, dtype=torch.bfloat16, device="cuda")
        buf[1:] = s[name].flatten()
        s[name] = buf[1:].view(s[name].shape)
    check_forward(far, s, "half", "misaligned")
    check_backward(far, s, "half", "misaligned")
    s = make(9, 3, 2, 128, 128, "bf16")
    buf = torch.empty(s["table"].numel() + 1, device="cuda")
    buf[1:] = s["table"].flatten()
    s["table"] = buf[1:].view(s["table"].shape)
    check_forward(far, s, "inter", "table off")
    check_backward(far, s, "inter", "table off")


def test_backward_in_place(far):
    """dq written over q, dk over dk_out."""
    s = make(21, 4, 2, 128, 64, "bf16")
    want = far.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"], s["pos"])
    q, dk = s["q"].clone(), s["dk"].clone()
    got = far.qk_norm_rope_backward(s["dq"], dk, q, s["k"], s["qw"], s["kw"], s["eps"], s["table"], s["pos"], dq=q, dk=dk)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_far_offsets(far):
    """Token strides past 2^32 bytes."""
    s = make(3, 2, 1, 128, 128, "bf16")
    stride = (1 << 31) + 8
    big = torch.empty(2 * stride + 256, dtype=torch.bfloat16, device="cuda")
    view = big.as_strided((3, 2, 128), (stride, 128, 1))
    view.copy_(s["q"])
    y, _ = far.qk_norm_rope(view, None, s["qw"], None, s["eps"], s["table"], s["pos"], q_out=view)
    within(y, *forward(s["q"], s["qw"], s["eps"], s["table"], s["pos"], "half"), "far offsets")


# ---------------------------------------------------------------------------
# positions and values
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dim", [128, 66])
def test_padding_tokens(far, dim):
    """Negative positions: zero rows whatever stands there (NaN too), zero gradients, nothing added."""
    s = make(12, 3, 1, dim, dim, "bf16")
    s["pos"][[0, 5, 11]] = torch.tensor([-1, -7, -(1 << 40)], device="cuda")
    for x in ("q", "k", "dq", "dk"):
        s[x][5] = float("nan")
    y, yk = far.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"], s["pos"])
    dq, dk, dqw, dkw = far.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"],
                                                 s["pos"])
    assert far.device_status() == 0
    for t in (y, yk, dq, dk):
        assert (t[[0, 5, 11]] == 0).all()
    for x in ("q", "k", "dq", "dk"):
        s[x][5] = 1.0
    for x, w, o, g, dx, dw in ((s["q"], s["qw"], y, s["dq"], dq, dqw), (s["k"], s["kw"], yk, s["dk"], dk, dkw)):
        within(o, *forward(x, w, s["eps"], s["table"], s["pos"], "half"), "padding")
        rdx, ex, rdw, ew = backward(g, x, w, s["eps"], s["table"], s["pos"], "half")
        within(dx, rdx, ex, "padding dx")
        within(dw, rdw, ew, "padding dw")


@pytest.mark.parametrize("dim", [128, 66])
def test_position_past_the_table(far, dim):
    """NaN rows and FAR_ERR_POSITION, once; the other rows right; nothing read past the table."""
    s = make(8, 3, 1, dim, dim, "bf16", rows=64)
    good = far.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"], s["pos"])
    pos = s["pos"].clone()
    pos[3], pos[6] = 64, 1 << 50
    got = far.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"], pos)
    assert far.device_status() == 11 and far.device_status() == 0
    keep = torch.tensor([0, 1, 2, 4, 5, 7], device="cuda")
    for a, b in zip(got, good):
        assert a[[3, 6]].isnan().all() and torch.equal(a[keep], b[keep])
    dq, _, dw, _ = far.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"], pos)
    assert far.device_status() == 11
    assert dq[[3, 6]].isnan().all() and not dq[keep].isnan().any() and not dw.isnan().any()


def test_special_values(far):
    """Zero heads (eps decides), tiny and huge heads, a NaN and an infinity: they stay in their head."""
    s = make(6, 2, 0, 128, 64, "f32")
    q = s["q"]
    q[0, 0] = 0.0
    q[1, 0] = 1e-20
    q[2, 0, 5] = float("nan")
    q[3, 0, 100] = float("inf")
    y, _ = far.qk_norm_rope(q, None, s["qw"], None, s["eps"], s["table"], s["pos"])
    assert (y[0, 0] == 0).all()
    assert y[2, 0].isnan().all() and y[3, 0, 100].isnan()
    rest = torch.ones(6, 2, dtype=torch.bool, device="cuda")
    rest[2, 0] = rest[3, 0] = False
    ref, err = forward(q, s["qw"], s["eps"], s["table"], s["pos"], "half")
    within(y[rest], ref[rest], err[rest], "special values")
    # the rotation alone: a value outside the rotated part is copied bit for bit, beside any other
    y, _ = far.rope(q, None, s["table"], s["pos"])
    assert torch.equal(y[..., 64:][rest], q[..., 64:][rest]) and math.isinf(float(y[3, 0, 100]))
    assert not y[3, 0, :64].isnan().any() and int(y[2, 0].isnan().sum()) == 2


def test_zero_eps_and_empty(far):
    s = make(4, 2, 1, 64, 64, "bf16")
    s["eps"] = 0.0
    check_forward(far, s, "half", "eps 0")
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    p = torch.empty(0, dtype=torch.int64, device="cuda")
    y, yk = far.qk_norm_rope(e, e, s["qw"], s["kw"], 1e-6, s["table"], p)
    assert y.shape == yk.shape == e.shape
    dq, _, dw, dkw = far.qk_norm_rope_backward(e, e, e, e, s["qw"], s["kw"], 1e-6, s["table"], p)
    assert (dw == 0).all() and (dkw == 0).all()


# ---------------------------------------------------------------------------
# streams, graphs, repetition
# ---------------------------------------------------------------------------

def test_same_bits_every_run(far):
    s = make(700, 8, 2, 128, 128, "bf16")
    call = lambda: far.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"],  # noqa: E731
                                             s["pos"])
    first = call()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(call(), first))


def test_streams_side_by_side(far):
    s = make(512, 8, 2, 128, 128, "bf16")
    args = (s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["table"], s["pos"])
    want, back = far.qk_norm_rope(*args), far.qk_norm_rope_backward(s["dq"], s["dk"], *args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(12):
        st = streams[i % 3]
        got.append(far.qk_norm_rope(*args, stream=st) + far.qk_norm_rope_backward(s["dq"], s["dk"], *args, stream=st))
    for st in streams:
        torch.cuda.current_stream().wait_stream(st)
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want + back))


def test_graph_capture_and_replay(far):
    s = make(64, 8, 2, 128, 128, "bf16")
    q, pos = s["q"].clone(), s["pos"].clone()
    run = lambda: far.qk_norm_rope(q, s["k"], s["qw"], s["kw"], s["eps"], s["table"], pos) + \
        far.qk_norm_rope_backward(s["dq"], s["dk"], q, s["k"], s["qw"], s["kw"], s["eps"], s["table"], pos)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(run())
    for seed in (5, 6):
        n = make(64, 8, 2, 128, 128, "bf16", seed=seed)
        q.copy_(n["q"])
        pos.copy_(n["pos"])
        for g in graphs:
            g.replay()
        want = run()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, want))


# ---------------------------------------------------------------------------
# the table
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("first", [0, 1000003])
@pytest.mark.parametrize("scaling", [None, {"type": "yarn", "factor": 4.0, "trained": 4096}])
def test_table(far, scaling, first):
    """Each value the binary32 rounding of the binary64 one: within half a step and the 2 units
    of binary64 that two sine routines may differ by (1e-9 relative to one, at angles to 10^6)."""
    rot, rows = 96, 3001
    freq, factor = far.rope_frequencies(rot, 1e4, scaling)
    t = far.rope_table(rows, rot, 1e4, scaling, first_position=first).cpu().numpy().astype(np.float64)
    angle = (first + np.arange(rows, dtype=np.float64))[:, None] * np.array(freq)
    want = np.concatenate([np.cos(angle), np.sin(angle)], 1) * factor
    assert (np.abs(t - want) <= 2.0 ** -24 * np.abs(want) + 1e-9 * factor).all()
    assert far.rope_table(0, 8).shape == (0, 8)
