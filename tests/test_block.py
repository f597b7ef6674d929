"""The 128-block FP8 operators without a GPU: refusals of the C entry points and the binding."""
import math

import pytest
import torch

A, MB = 1 << 40, 1 << 20  # stand-in addresses: validated, never read


@pytest.fixture(scope="module")
def far():
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    return far


def norm(far, **kw):
    d = dict(x=A, xs=512, r=A + MB, rs=512, w=A + 2 * MB, eps=1e-6, q=A + 3 * MB, s=A + 4 * MB, ro=A + 5 * MB, ros=512, n=4,
             h=512, dt=0x22)
    d.update(kw)
    return far.lib.fused_add_rmsnorm_quant_block(d["x"], d["xs"], d["r"], d["rs"], d["w"], d["eps"], d["q"], d["s"], d["ro"],
                                                 d["ros"], d["n"], d["h"], d["dt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=0x12), 1), (dict(dt=0x32), 2), (dict(eps=-1.0), 6), (dict(eps=math.nan), 6), (dict(h=0), 4), (dict(n=-1), 4),
    (dict(xs=511), 4), (dict(ros=500), 4), (dict(x=None), 3), (dict(r=None), 3), (dict(w=None), 3), (dict(q=None), 3),
    (dict(s=None), 3), (dict(ro=None), 3), (dict(q=A), 5), (dict(q=A + MB), 5), (dict(s=A + 3 * MB + 8), 5),
    (dict(s=A + 5 * MB - 60), 5),  # 4 rows x 4 blocks x 4 bytes: past what one scale a row would take
    (dict(ro=A + 2), 5), (dict(s=A), 5), (dict(s=A + 2 * MB), 5)])
def test_norm_refusals(far, kw, status):
    assert norm(far, **kw) == status


@pytest.mark.parametrize("kw", [dict(x=A + 1), dict(r=A + MB + 1), dict(w=A + 2 * MB + 1), dict(ro=A + 5 * MB + 1),
                                dict(s=A + 4 * MB + 2), dict(w=A + 2 * MB + 2, dt=0x02)])
def test_norm_misaligned_elements(far, kw):
    assert norm(far, **kw) == 4


def test_norm_nothing_to_do(far):
    assert norm(far, n=0, x=None, r=None, q=None, s=None, ro=None) == 0
    assert far.lib.rmsnorm_quant_block(A, 512, A + MB, 1e-6, A + 2 * MB, None, 4, 512, 0x22, None) == 3
    assert far.lib.rmsnorm_quant_block(A, 511, A + MB, 1e-6, A + 2 * MB, A + 3 * MB, 4, 512, 0x22, None) == 4


def quant(far, **kw):
    d = dict(x=A, xs=256, q=A + MB, s=A + 2 * MB, r=256, c=256, block=0, t=0, act=2)
    d.update(kw)
    return far.lib.quant_block_fp8(d["x"], d["xs"], d["q"], d["s"], d["r"], d["c"], d["block"], d["t"], d["act"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(act=3), 2), (dict(act=-1), 2), (dict(block=2), 2), (dict(block=-1), 2), (dict(t=2), 2), (dict(r=-1), 4),
    (dict(c=-1), 4), (dict(xs=255), 4), (dict(r=1 << 32), 4), (dict(x=None), 3), (dict(q=None), 3), (dict(s=None), 3),
    (dict(x=A + 1), 4), (dict(s=A + 2 * MB + 2), 4), (dict(q=A + 100), 5), (dict(q=A + 2 * MB), 5), (dict(s=A + 1000), 5),
    (dict(s=A + MB + 65532), 5), (dict(r=0, x=None), 0), (dict(c=0, q=None), 0)])
def test_quant_refusals(far, kw, status):
    assert quant(far, **kw) == status


def gemm(far, **kw):
    d = dict(x=A, ldx=256, xs=A + MB, w=A + 2 * MB, ldw=256, ws=A + 3 * MB, block=1, out=A + 4 * MB, ldo=128, m=4, n=128, k=256,
             od=2)
    d.update(kw)
    return far.lib.gemm_fp8_block(d["x"], d["ldx"], d["xs"], d["w"], d["ldw"], d["ws"], d["block"], d["out"], d["ldo"], d["m"],
                                  d["n"], d["k"], d["od"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(od=3), 2), (dict(od=-1), 2), (dict(block=2), 2), (dict(m=-1), 4), (dict(n=-1), 4), (dict(k=-1), 4),
    (dict(m=1 << 31), 4), (dict(ldx=255), 4), (dict(ldw=255), 4), (dict(ldo=127), 4), (dict(x=None), 3), (dict(w=None), 3),
    (dict(xs=None), 3), (dict(ws=None), 3), (dict(out=None), 3), (dict(out=A + 4 * MB + 1), 4), (dict(xs=A + MB + 2), 4),
    (dict(ws=A + 3 * MB + 1), 4), (dict(out=A), 5), (dict(out=A + 2 * MB + 30000), 5), (dict(out=A + MB), 5),
    (dict(out=A + 3 * MB - 512), 5), (dict(m=0, x=None, out=None), 0), (dict(n=0, ldo=0, out=None), 0)])
def test_gemm_refusals(far, kw, status):
    assert gemm(far, **kw) == status


def test_binding_refusals(far):
    x = torch.zeros(4, 256)
    w = torch.ones(256)
    q, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    for call, text in ((lambda: far.rmsnorm_quant_block(x, w, 1e-6), "CUDA"),
                       (lambda: far.rmsnorm_quant_block(x, w[:8], 1e-6), "weight"),
                       (lambda: far.fused_add_rmsnorm_quant_block(x, x[:2], w, 1e-6), "share"),
                       (lambda: far.quant_block_fp8(w), "matrix"),
                       (lambda: far.quant_block_fp8(x, block="cols"), "block"),
                       (lambda: far.quant_block_fp8(x), "CUDA"),
                       (lambda: far.gemm_fp8_block(x, s, q, s), "codes"),
                       (lambda: far.gemm_fp8_block(q, s, q[:, :128], s), r"\[n, k\]"),
                       (lambda: far.gemm_fp8_block(q, s[:, :1], q, s), "x_scale"),
                       (lambda: far.gemm_fp8_block(q, s, q, s[:3]), "wt_scale"),
                       (lambda: far.gemm_fp8_block(q, s, q, s.double()), "wt_scale"),
                       (lambda: far.gemm_fp8_block(q, s, q, s), "CUDA")):
        with pytest.raises(ValueError, match=text):
            call()
    with pytest.raises(far.FarError):
        far.quant_block_fp8(x.double())
    with pytest.raises(far.FarError):
        far.gemm_fp8_block(q, s, q, s, out_dtype=torch.float64)


def test_gemm_plans(far):
    """Decode batches and few rows take the small kernel with k shared out while SMs are free, large
    products CTA pairs, k that TMA cannot step over the plain kernel."""
    plan = far.plan_gemm_fp8_for_sms
    assert plan(1, 8192, 8192, "tile", 152) == {"kind": 2, "rows": 16, "split": 4, "grid": 256}
    assert plan(17, 8192, 8192, "row", 152)["rows"] == 32 and plan(33, 8192, 8192, "tile", 152)["rows"] == 64
    assert plan(4, 1024, 8192, "tile", 152)["split"] == 8
    assert plan(4, 128, 384, "tile", 152)["split"] == 1  # three blocks of k are not shared out
    assert plan(128, 8192, 8192, "tile", 152)["kind"] == 2 and plan(192, 8192, 8192, "tile", 152)["kind"] == 1
    assert plan(16384, 8192, 8192, "tile", 152) == {"kind": 1, "rows": 0, "split": 0, "grid": 152}
    assert plan(600, 777, 640, "tile", 152)["kind"] == 1 and plan(3000, 1102, 256, "row", 152)["kind"] == 1
    assert plan(4, 128, 1000, "tile", 152)["kind"] == 0 and plan(16384, 8192, 100, "tile", 152)["kind"] == 0
    assert plan(1 << 30, 1 << 30, 128, "tile", 152)["kind"] == 0  # more tiles than are counted
    for m, n, k in ((1, 1, 16), (64, 100000, 128), (2000000, 128, 4096), (1, 1 << 23, 256)):
        p = plan(m, n, k, "tile", 152)
        assert p["kind"] in (1, 2) and p["grid"] >= 1
        if p["kind"] == 2:  # no CTA without a block of k, clusters of a portable size
            assert p["split"] <= 8 and p["split"] <= -(-k // 128)
    for bad in ((0, 8, 8), (8, 0, 8), (8, 8, 0), (1 << 31, 8, 8)):
        with pytest.raises(far.FarError):
            plan(*bad, "tile", 152)
