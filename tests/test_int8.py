"""quant_rows_int8 and gemm_int8 without a GPU: refusals of the C entry points and the binding."""
import pytest
import torch

A, MB = 1 << 40, 1 << 20  # stand-in addresses: validated, never read


@pytest.fixture(scope="module")
def far():
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    return far


def quant(far, **kw):
    d = dict(x=A, xs=256, q=A + MB, s=A + 2 * MB, r=256, c=256, act=2)
    d.update(kw)
    return far.lib.quant_rows_int8(d["x"], d["xs"], d["q"], d["s"], d["r"], d["c"], d["act"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(act=3), 2), (dict(act=-1), 2), (dict(r=-1), 4), (dict(c=-1), 4), (dict(xs=255), 4), (dict(r=1 << 31), 4),
    (dict(x=None), 3), (dict(q=None), 3), (dict(s=None), 3), (dict(c=0, s=None), 3), (dict(x=A + 1), 4),
    (dict(x=A + 2, act=0), 4), (dict(s=A + 2 * MB + 2), 4), (dict(q=A + 100), 5), (dict(q=A + 2 * MB), 5),
    (dict(s=A + 512), 5), (dict(s=A + MB + 65532), 5), (dict(r=0, x=None, q=None, s=None), 0)])
def test_quant_refusals(far, kw, status):
    assert quant(far, **kw) == status


def gemm(far, **kw):
    d = dict(x=A, ldx=256, xs=A + MB, w=A + 2 * MB, ldw=256, ws=A + 3 * MB, b=A + 4 * MB, out=A + 5 * MB, ldo=128,
             space=None, bytes=0, m=4, n=128, k=256, od=2)
    d.update(kw)
    return far.lib.gemm_int8(d["x"], d["ldx"], d["xs"], d["w"], d["ldw"], d["ws"], d["b"], d["out"], d["ldo"], d["space"],
                             d["bytes"], d["m"], d["n"], d["k"], d["od"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(od=3), 2), (dict(od=-1), 2), (dict(m=-1), 4), (dict(n=-1), 4), (dict(k=-1), 4), (dict(m=1 << 31), 4),
    (dict(k=131072, ldx=1 << 18, ldw=1 << 18), 4), (dict(ldx=255), 4), (dict(ldw=255), 4), (dict(ldo=127), 4),
    (dict(x=None), 3), (dict(w=None), 3), (dict(xs=None), 3), (dict(ws=None), 3), (dict(out=None), 3),
    (dict(k=0, xs=None), 3), (dict(out=A + 5 * MB + 1), 4), (dict(b=A + 4 * MB + 1), 4), (dict(od=0, b=A + 4 * MB + 2), 4),
    (dict(xs=A + MB + 2), 4), (dict(ws=A + 3 * MB + 1), 4), (dict(out=A), 5), (dict(out=A + 2 * MB + 30000), 5),
    (dict(out=A + MB), 5), (dict(out=A + 3 * MB - 512), 5), (dict(out=A + 4 * MB - 16), 5),
    (dict(m=0, x=None, out=None), 0), (dict(n=0, ldo=0, out=None), 0)])
def test_gemm_refusals(far, kw, status):
    assert gemm(far, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(space=None), 9), (dict(bytes=6 * MB - 1), 9), (dict(space=A + 64 * MB + 8), 9), (dict(space=A), 5),
    (dict(space=A + 5 * MB - 4096), 5)])
def test_gemm_workspace_refusals(far, kw, status):
    """Many rows: x as f16 and room for wt's codes, (2 m + n) k bytes."""
    m, n, k = 2048, 2048, 1024
    assert far.gemm_int8_workspace_bytes(m, n, k) == (2 * m + n) * k and far.plan_gemm_int8(m, n, k)["kind"] == 1
    d = dict(x=A, w=A + 16 * MB, xs=A + 32 * MB, ws=A + 33 * MB, b=None, out=A + 5 * MB, ldo=n, space=A + 64 * MB, bytes=6 * MB,
             m=m, n=n, k=k, ldx=k, ldw=k)
    d.update(kw)
    assert gemm(far, **d) == status


def test_plans(far):
    """Few rows a cluster of CTAs, as many as share k and fit at once; many rows CTA pairs, where their tiles fill them."""
    plan = far.plan_gemm_int8
    assert plan(1, 8192, 8192) == {"kind": 2, "rows": 16, "split": 4}
    assert plan(16, 5120, 5120)["split"] == 6  # clusters of 7 do not all fit
    assert plan(17, 8192, 8192)["rows"] == 32 and plan(64, 512, 8192)["rows"] == 64 and plan(65, 512, 8192)["rows"] == 128
    assert plan(128, 8192, 8192) == {"kind": 2, "rows": 128, "split": 2}
    assert plan(777, 512, 8192)["kind"] == 2 and plan(300, 512, 2048)["kind"] == 2
    assert plan(200, 5120, 13312)["kind"] == 1 and plan(777, 2056, 4112) == {"kind": 1, "rows": 128, "split": 0}
    assert plan(16384, 8192, 8192) == {"kind": 1, "rows": 192, "split": 0}
    assert plan(1, 1, 16) == {"kind": 2, "rows": 16, "split": 1}
    assert plan(1, 1, 1)["kind"] == 0 and plan(4, 1000, 20)["kind"] == 0  # k that TMA cannot step over:
    assert plan(4, 8192, 8191)["kind"] == 1 and plan(400, 1000, 3000)["kind"] == 1  # plain while short, else repacked
    assert plan(2 ** 31 - 1, 2 ** 31 - 1, 64)["kind"] == 0  # more tiles than are counted
    for m, n, k in ((1, 1 << 30, 128), (1 << 30, 1, 128), (5000, 5000, 131071)):
        plan(m, n, k)
        far.gemm_int8_workspace_bytes(m, n, k)
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 131072)):
        with pytest.raises(far.FarError):
            plan(*bad)


def test_workspace_sizes(far):
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, -1), (1, 1, 131072), (1 << 31, 1, 1)):
        with pytest.raises(far.FarError):
            far.gemm_int8_workspace_bytes(*bad)
    assert far.gemm_int8_workspace_bytes(0, 0, 0) == 0


def test_binding_refusals(far):
    q, w = torch.zeros(4, 256, dtype=torch.int8), torch.zeros(8, 256, dtype=torch.int8)
    s, ws = torch.ones(4), torch.ones(8)
    for call, text in ((lambda: far.gemm_int8(q.float(), s, w, ws), "codes"),
                       (lambda: far.gemm_int8(q, s, w[:, :128], ws), r"\[n, k\]"),
                       (lambda: far.gemm_int8(q, s[:3], w, ws), "x_scale"),
                       (lambda: far.gemm_int8(q, s.double(), w, ws), "x_scale"),
                       (lambda: far.gemm_int8(q, s, w, ws[:, None]), "wt_scale"),
                       (lambda: far.gemm_int8(q, s, w, ws, torch.ones(8)), "bias"),
                       (lambda: far.gemm_int8(q, s, w, ws), "CUDA"),
                       (lambda: far.quant_rows_int8(s), "CUDA"),
                       (lambda: far.quant_rows_int8(torch.tensor(1.0)), "cols")):
        with pytest.raises(ValueError, match=text):
            call()
    with pytest.raises(far.FarError):
        far.quant_rows_int8(s.double())
    with pytest.raises(far.FarError):
        far.gemm_int8(q, s, w, ws, out_dtype=torch.float64)
    with pytest.raises(TypeError):
        far.gemm_int8(q, s, w, ws, out_dtype="bf16")
    with pytest.raises(TypeError):
        far.gemm_int8(q, None, w, ws)
