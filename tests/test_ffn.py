"""gated_ffn and its gradients without a GPU: refusals of the C entry points and the binding, and the
reference's own derivatives against differences."""
import pytest
import torch

import ffn_ref as ref

A, MB = 1 << 40, 1 << 20  # stand-in addresses: validated, never read


@pytest.fixture(scope="module")
def far():
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    return far


def gate(far, **kw):
    d = dict(x=A, ldx=256, wg=A + MB, ldg=256, wu=A + 2 * MB, ldu=256, out=A + 3 * MB, ldo=512, go=A + 4 * MB, ldgo=512,
             uo=A + 5 * MB, lduo=512, m=4, h=256, f=512, act=0, dt=2)
    d.update(kw)
    return far.lib.gated_ffn(d["x"], d["ldx"], d["wg"], d["ldg"], d["wu"], d["ldu"], d["out"], d["ldo"], d["go"], d["ldgo"],
                             d["uo"], d["lduo"], d["m"], d["h"], d["f"], d["act"], d["dt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=0), 2), (dict(dt=3), 2), (dict(act=3), 2), (dict(act=-1), 2), (dict(m=-1), 4), (dict(h=-1), 4), (dict(f=-1), 4),
    (dict(m=1 << 31), 4), (dict(ldx=255), 4), (dict(ldg=255), 4), (dict(ldu=255), 4), (dict(ldo=511), 4), (dict(ldgo=511), 4),
    (dict(lduo=511), 4), (dict(ldx=(1 << 31) + 1), 4), (dict(x=None), 3), (dict(wg=None), 3), (dict(wu=None), 3),
    (dict(out=None), 3), (dict(go=None), 3), (dict(uo=None), 3), (dict(x=A + 1), 4), (dict(wu=A + 2 * MB + 1), 4),
    (dict(out=A + 3 * MB + 1), 4), (dict(go=A + 4 * MB + 1), 4), (dict(out=A), 5), (dict(out=A + MB + 512), 5),
    (dict(go=A + 2 * MB), 5), (dict(uo=A + 3 * MB), 5), (dict(uo=A + 4 * MB - 2), 5), (dict(m=0, x=None, out=None), 0),
    (dict(f=0, wg=None), 0)])
def test_forward_refusals(far, kw, status):
    assert gate(far, **kw) == status


def back(far, **kw):
    d = dict(dh=A, lddh=512, g=A + MB, ldg=512, u=A + 2 * MB, ldu=512, x=A + 3 * MB, ldx=256, wg=A + 4 * MB, ldwg=256,
             wu=A + 5 * MB, ldwu=256, dx=A + 6 * MB, lddx=256, dwg=A + 7 * MB, lddwg=256, dwu=A + 8 * MB, lddwu=256,
             ws=A + 9 * MB, wsb=MB, m=4, h=256, f=512, act=0, dt=2)
    d.update(kw)
    return far.lib.gated_ffn_backward(d["dh"], d["lddh"], d["g"], d["ldg"], d["u"], d["ldu"], d["x"], d["ldx"], d["wg"],
                                      d["ldwg"], d["wu"], d["ldwu"], d["dx"], d["lddx"], d["dwg"], d["lddwg"], d["dwu"],
                                      d["lddwu"], d["ws"], d["wsb"], d["m"], d["h"], d["f"], d["act"], d["dt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=0), 2), (dict(act=7), 2), (dict(m=-1), 4), (dict(f=1 << 31), 4), (dict(lddh=511), 4), (dict(lddx=255), 4),
    (dict(lddwu=255), 4), (dict(dh=None), 3), (dict(u=None), 3), (dict(dx=None), 3), (dict(dwg=None), 3), (dict(dwu=None), 3),
    (dict(g=A + MB + 1), 4), (dict(dwg=A + 7 * MB + 1), 4), (dict(dx=A), 5), (dict(dwg=A + 6 * MB), 5),
    (dict(dwu=A + 7 * MB + 1024), 5), (dict(dwu=A + 5 * MB), 5), (dict(ws=None), 9), (dict(wsb=8191), 9),
    (dict(ws=A + 9 * MB + 8), 9), (dict(ws=A), 5), (dict(ws=A + 6 * MB + 64), 5), (dict(ws=A + 8 * MB - 16), 5),
    (dict(h=0, x=None, dx=None), 0)])
def test_backward_refusals(far, kw, status):
    assert back(far, **kw) == status


def test_plans(far):
    """Up to 64 tokens always a cluster of CTAs a tile; more by estimate; many tokens CTA pairs."""
    plan = far.plan_gated_ffn
    assert plan(1, 5120, 13312) == {"kind": 2, "tokens": 16, "split": 1}
    assert plan(60, 2056, 5640) == {"kind": 2, "tokens": 64, "split": 3}
    assert plan(1, 1024, 1024)["split"] == 8 and plan(1, 64, 64) == {"kind": 2, "tokens": 16, "split": 1}
    assert plan(200, 5120, 512)["kind"] == 2 and plan(200, 2048, 5632)["kind"] == 1
    assert plan(8192, 5120, 13312) == {"kind": 1, "tokens": 0, "split": 0}
    assert plan(2 ** 31 - 1, 8, 2 ** 31 - 1)["kind"] == 0  # more tiles than are counted
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 31, 1, 1)):
        with pytest.raises(far.FarError):
            plan(*bad)


def test_workspace_sizes(far):
    assert far.gated_ffn_backward_workspace_bytes(4, 512) == 8192
    assert far.gated_ffn_backward_workspace_bytes(3, 5) == 3 * 8 * 4  # rows of whole 16 bytes
    assert far.gated_ffn_backward_workspace_bytes(0, 5) == 0
    for bad in ((-1, 5), (5, -1), (1 << 31, 5), (5, 1 << 31)):
        with pytest.raises(far.FarError):
            far.gated_ffn_backward_workspace_bytes(*bad)


def test_binding_refusals(far):
    x, w, h = torch.zeros(4, 256).half(), torch.zeros(32, 256).half(), torch.zeros(4, 32).half()
    for call, text in ((lambda: far.gated_ffn(x, w, w, activation="relu"), "activation"),
                       (lambda: far.gated_ffn(x, w, w[:16]), "hidden"),
                       (lambda: far.gated_ffn(x[:, :8], w, w), "hidden"),
                       (lambda: far.gated_ffn(x[0], w, w), "hidden"),
                       (lambda: far.gated_ffn(x, w.bfloat16(), w), "dtype"),
                       (lambda: far.gated_ffn(x, w, w, gate_out=h), "save"),
                       (lambda: far.gated_ffn(x, w, w), "CUDA"),
                       (lambda: far.gated_ffn_backward(h, h, h[:2], x, w, w), "ffn"),
                       (lambda: far.gated_ffn_backward(h, h.float(), h, x, w, w), "dtype"),
                       (lambda: far.gated_ffn_backward(h, h, h, x, w, w), "CUDA")):
        with pytest.raises(ValueError, match=text):
            call()
    with pytest.raises(far.FarError):
        far.gated_ffn(x.float(), w.float(), w.float())


@pytest.mark.parametrize("name", ref.ACTS)
def test_reference_against_differences(name):
    """The reference's slopes and gradients, by central differences in 64 bits (error d^2 / 6 of third derivatives)."""
    g = torch.linspace(-9, 9, 301, dtype=torch.float64)
    d = 1e-5
    assert torch.allclose(ref.slope(g, name), (ref.act(g + d, name) - ref.act(g - d, name)) / (2 * d), atol=1e-9, rtol=0)
    rng = torch.Generator().manual_seed(1)
    x, wg, wu, c = (torch.randn(*s, generator=rng, dtype=torch.float64) / 2 for s in ((3, 5), (4, 5), (4, 5), (3, 4)))

    def loss(x, wg, wu):
        return (c * ref.act(x @ wg.T, name) * (x @ wu.T)).sum()

    gate, up = x @ wg.T, x @ wu.T
    dg, du = c * up * ref.slope(gate, name), c * ref.act(gate, name)
    grads = [dg @ wg + du @ wu, dg.T @ x, du.T @ x]
    leaves = [x, wg, wu]
    for n, grad in enumerate(grads):
        for i in range(leaves[n].numel()):
            e = torch.zeros_like(leaves[n]).view(-1)
            e[i] = d
            e = e.view_as(leaves[n])
            up_, down = (loss(*[v + s * e if k == n else v for k, v in enumerate(leaves)]) for s in (1, -1))
            assert abs(float((up_ - down) / (2 * d) - grad.view(-1)[i])) < 1e-8
