"""The per-head norm and rotation without a GPU: refusals of the C entry points and of the
binding, and the rotation frequencies against their definitions.  No call here reaches CUDA."""
import ctypes
import math

import pytest
import torch

A = 1 << 40  # stand-in addresses: validated, never read
MB = 1 << 20


@pytest.fixture(scope="module")
def far():
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    return far


def call(far, back=False, **kw):
    """qk_norm_rope (or its backward) on stand-in addresses: 4 tokens, 2 + 1 heads of 64, bf16."""
    d = dict(q=A, qts=128, qhs=64, k=A + MB, kts=64, khs=64, qw=A + 2 * MB, kw=A + 3 * MB, eps=1e-6, table=A + 4 * MB,
             rows=16, pos=A + 5 * MB, pb=8, yq=A + 6 * MB, yqts=128, yqhs=64, yk=A + 7 * MB, ykts=64, ykhs=64,
             gq=A + 8 * MB, gk=A + 9 * MB, dqw=A + 10 * MB, dkw=A + 11 * MB, ws=A + 16 * MB, wsb=8 * MB,
             tokens=4, h=2, hk=1, dim=64, rot=64, pairs=0, dtype=0x22)
    d.update(kw)
    xs = (d["q"], d["qts"], d["qhs"], d["k"], d["kts"], d["khs"])
    place = (d["table"], d["rows"], d["pos"], d["pb"])
    ys = (d["yq"], d["yqts"], d["yqhs"], d["yk"], d["ykts"], d["ykhs"])
    sizes = (d["tokens"], d["h"], d["hk"], d["dim"], d["rot"], d["pairs"], d["dtype"])
    if not back:
        return far.lib.qk_norm_rope(*xs, d["qw"], d["kw"], d["eps"], *place, *ys, *sizes, None)
    return far.lib.qk_norm_rope_backward(d["gq"], 128, 64, d["gk"], 64, 64, *xs, d["qw"], d["kw"], d["eps"], *place, *ys,
                                         d["dqw"], d["dkw"], d["ws"], d["wsb"], *sizes, None)


REFUSED = [
    (dict(dtype=0x12), 1), (dict(dtype=0x21), 1), (dict(dtype=0x23), 2), (dict(dtype=0x122), 2), (dict(dtype=-1), 2),
    (dict(pb=2), 2), (dict(pairs=2), 2), (dict(pairs=-1), 2),
    (dict(eps=-1e-6), 6), (dict(eps=math.nan), 6), (dict(eps=math.inf), 6),
    (dict(tokens=-1), 4), (dict(h=-1), 4), (dict(dim=0), 4), (dict(dim=2049, rot=64), 4), (dict(rot=63), 4),
    (dict(rot=0), 4), (dict(rot=66), 4), (dict(rows=0), 4), (dict(rows=-1), 4), (dict(tokens=1 << 32), 4),
    (dict(qts=-128), 4), (dict(yqts=1 << 50), 4),
    (dict(yqhs=0), 4), (dict(yqts=64), 4), (dict(yqhs=63), 4),  # two outputs in one place
    (dict(q=A + 1), 4), (dict(pos=A + 5 * MB + 4), 4), (dict(table=A + 4 * MB + 2), 4),  # element alignment
    (dict(q=None), 3), (dict(k=None), 3), (dict(qw=None), 3), (dict(kw=None), 3), (dict(table=None), 3),
    (dict(pos=None), 3), (dict(yq=None), 3), (dict(yk=None), 3),
    (dict(yq=A + 2), 5), (dict(yq=A, yqts=256), 5), (dict(yq=A + MB), 5), (dict(yk=A), 5), (dict(yk=A + 6 * MB + 64), 5),
    (dict(yq=A + 2 * MB), 5), (dict(yq=A + 4 * MB), 5), (dict(yk=A + 5 * MB), 5),
]


@pytest.mark.parametrize("kw,status", REFUSED)
def test_forward_refusals(far, kw, status):
    assert call(far, **kw) == status


@pytest.mark.parametrize("kw,status", REFUSED + [
    (dict(gq=None), 3), (dict(gk=None), 3), (dict(dqw=None), 3), (dict(dkw=None), 3),
    (dict(ws=None), 9), (dict(wsb=1024 * 64 * 4 - 1), 9), (dict(ws=A + 16 * MB + 8), 9),
    (dict(yq=A + 8 * MB + 2), 5), (dict(yq=A + 9 * MB), 5), (dict(dqw=A + 6 * MB), 5), (dict(dqw=A + 11 * MB + 128), 5),
    (dict(dkw=A), 5), (dict(ws=A + 8 * MB), 5), (dict(ws=A + 10 * MB - 64), 5)])
def test_backward_refusals(far, kw, status):
    assert call(far, back=True, **kw) == status


def test_misaligned_weights(far):
    for back in (False, True):
        assert call(far, back=back, qw=A + 2 * MB + 1) == 4 and call(far, back=back, kw=A + 3 * MB + 1) == 4
        assert call(far, back=back, kw=A + 3 * MB + 2, dtype=0x02) == 4
    assert call(far, back=True, dqw=A + 10 * MB + 2) == 4 and call(far, back=True, dkw=A + 11 * MB + 1) == 4


def test_head_count_refusals(far):
    for back in (False, True):
        assert call(far, back=back, tokens=0, h=(1 << 30) + 1) == 4 and call(far, back=back, tokens=0, hk=(1 << 30) + 1) == 4
    assert call(far, tokens=0, h=1 << 30, hk=1 << 30) == 0


def test_rope_refusals(far):
    def rope(transpose=0, act=2, q=A, y=A + MB):
        return far.lib.rope(q, 64, 64, None, 0, 0, A + 4 * MB, 16, A + 5 * MB, 8, y, 64, 64, None, 0, 0, 4, 1, 0, 64, 64,
                            0, transpose, act, None)

    assert rope(transpose=2) == 2 and rope(act=3) == 2 and rope(q=None) == 3 and rope(y=A + 64) == 5


def test_interleaved_views_in_place(far):
    """q and k interleaved head by head in one buffer: in place is allowed, a value's overlap is not."""
    il = dict(q=A, qts=768, qhs=192, k=A + 128, kts=768, khs=192, hk=2, yq=A, yqts=768, yqhs=192, yk=A + 128, ykts=768, ykhs=192)
    assert call(far, **{**il, "yk": A + 126}) == 5  # k_out one value into q's head
    assert call(far, **{**il, "yk": A + 128 + 64}) == 5  # between its own heads: shares bytes with k
    assert call(far, **{**il, "k": A + 128 + 768 * 2 * 3, "yk": A + 128 + 768 * 2 * 3 - 2}) == 5
    # (the allowed calls run on the GPU: test_gpu_heads.py)


def test_nothing_to_do(far):
    """No tokens, or no heads: accepted without touching anything."""
    assert call(far, tokens=0, q=None, k=None, yq=None, yk=None, pos=None, table=None, rows=0) == 0
    assert call(far, h=0, hk=0) == 0


def test_workspace_bytes(far):
    assert far.qk_backward_workspace_bytes(128) == 1024 * 128 * 4
    for bad in (0, -1, 2049):
        with pytest.raises(far.FarError):
            far.qk_backward_workspace_bytes(bad)


def test_binding_refusals(far):
    q, w, t, p = torch.zeros(4, 2, 64), torch.ones(64), torch.zeros(8, 64), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        far.qk_norm_rope(q, None, w, None, 1e-6, t, p)
    with pytest.raises(ValueError, match="head_dim"):
        far.rope(q[0], None, t, p)
    with pytest.raises(ValueError, match="agree"):
        far.qk_norm_rope(q, torch.zeros(3, 2, 64), w, w, 1e-6, t, p)
    with pytest.raises(ValueError, match="dtype"):
        far.qk_norm_rope(q, q.half(), w, w, 1e-6, t, p)
    with pytest.raises(ValueError, match="weight"):
        far.qk_norm_rope(q, q, w, w[:32], 1e-6, t, p)
    with pytest.raises(ValueError, match="weight"):
        far.qk_norm_rope(q, q, w, None, 1e-6, t, p)
    with pytest.raises(ValueError, match="gradient"):
        far.qk_norm_rope_backward(q[:, :1], None, q, None, w, None, 1e-6, t, p)
    with pytest.raises(ValueError, match="CUDA"):
        far.rope_table(8, 64, device="cpu")


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------

def plain(rot, base):
    return [base ** (-2 * j / rot) for j in range(rot // 2)]


def test_plain_linear_and_ntk(far):
    f, m = far.rope_frequencies(128, 1e6)
    assert m == 1.0 and f == pytest.approx(plain(128, 1e6), rel=1e-14)
    f, m = far.rope_frequencies(96, 1e4, {"type": "linear", "factor": 8.0})
    assert m == 1.0 and f == pytest.approx([v / 8 for v in plain(96, 1e4)], rel=1e-14)
    f, _ = far.rope_frequencies(64, 1e4, {"type": "ntk", "factor": 4.0})
    assert f[0] == 1.0  # the fastest pair is untouched, the slowest stretched by the factor
    assert f[-1] == pytest.approx(plain(64, 1e4)[-1] / 4.0, rel=1e-12)


def test_yarn(far):
    rot, base, a, trained = 128, 1e4, 4.0, 4096
    f, m = far.rope_frequencies(rot, base, {"type": "yarn", "factor": a, "trained": trained})
    p = plain(rot, base)
    assert m == pytest.approx(0.1 * math.log(a) + 1)
    ratio = [x / y for x, y in zip(f, p)]
    for j in range(rot // 2):
        turns = trained * p[j] / (2 * math.pi)
        if turns > 33:
            assert ratio[j] == pytest.approx(1.0, rel=1e-3)  # pairs of many turns keep their frequency
        if turns < 0.9:
            assert ratio[j] == pytest.approx(1 / a, rel=1e-12)  # pairs that never come round are stretched
    inner = [r for r in ratio if 1 / a + 1e-9 < r < 1 - 1e-9]
    assert inner and all(x > y for x, y in zip(inner, inner[1:]))
    step = [x - y for x, y in zip(inner, inner[1:])]
    assert step == pytest.approx([step[0]] * len(step), rel=1e-6)  # a straight ramp over the pairs between
    assert far.rope_frequencies(rot, base, {"type": "yarn", "factor": a, "trained": trained, "attention_factor": 1.25})[1] == 1.25
    assert far.rope_frequencies(rot, base, {"type": "yarn", "factor": 1.0, "trained": trained})[1] == 1.0


def test_bands(far):
    rot, base, a, trained = 128, 5e5, 8.0, 8192
    f, m = far.rope_frequencies(rot, base, {"type": "bands", "factor": a, "trained": trained, "low": 1.0, "high": 4.0})
    assert m == 1.0
    for x, y in zip(f, plain(rot, base)):
        wave = 2 * math.pi / y
        if wave < trained / 4.0:
            want = y
        elif wave > trained / 1.0:
            want = y / a
        else:
            s = (trained / wave - 1.0) / 3.0
            want = (1 - s) * y / a + s * y
        assert x == pytest.approx(want, rel=1e-12)


def test_frequency_refusals(far):
    L = far.lib
    buf = (ctypes.c_double * 64)()
    p, f, m = (ctypes.c_double * 5)(4.0, 4096.0, 32.0, 1.0, 0.0), ctypes.addressof(buf), ctypes.addressof(ctypes.c_double())
    pp = ctypes.addressof(p)
    assert L.far_rope_frequencies(0, 1e4, 0, pp, f, m) == 4 and L.far_rope_frequencies(63, 1e4, 0, pp, f, m) == 4
    assert L.far_rope_frequencies(4096, 1e4, 0, pp, f, m) == 4 and L.far_rope_frequencies(2, 1e4, 2, pp, f, m) == 4
    assert L.far_rope_frequencies(64, 1e4, 5, pp, f, m) == 2 and L.far_rope_frequencies(64, 1e4, 1, None, f, m) == 3
    assert L.far_rope_frequencies(64, 1.0, 0, pp, f, m) == 6 and L.far_rope_frequencies(64, math.inf, 0, pp, f, m) == 6
    p[0] = 0.0
    assert L.far_rope_frequencies(64, 1e4, 1, pp, f, m) == 6
    for bad in ({"type": "other"}, {"type": "linear"}, {"type": "linear", "factor": 2.0, "trained": 3}, {"type": "yarn", "factor": 2.0}):
        with pytest.raises(ValueError):
            far.rope_frequencies(64, 1e4, bad)


def test_table_refusals(far):
    f = (ctypes.c_double * 32)(*([1.0] * 32))
    a = ctypes.addressof(f)
    assert far.lib.rope_table(A, -1, 64, 0, a, 1.0, None) == 4 and far.lib.rope_table(A, 8, 63, 0, a, 1.0, None) == 4
    assert far.lib.rope_table(A, 8, 64, -1, a, 1.0, None) == 4 and far.lib.rope_table(A + 2, 8, 64, 0, a, 1.0, None) == 4
    assert far.lib.rope_table(None, 8, 64, 0, a, 1.0, None) == 3 and far.lib.rope_table(A, 8, 64, 0, None, 1.0, None) == 3
    assert far.lib.rope_table(A, 8, 64, 0, a, math.nan, None) == 6
    f[3] = math.inf
    assert far.lib.rope_table(A, 8, 64, 0, a, 1.0, None) == 6
    assert far.lib.rope_table(None, 0, 64, 0, ctypes.addressof((ctypes.c_double * 32)()), 1.0, None) == 0


def test_table_on_another_devices_stream(far):
    """refused before anything is made: a table asked for on one device, with a stream of another"""
    from types import SimpleNamespace

    stream = SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="another device"):
        far.rope_table(8, 64, device="cuda:0", stream=stream)
