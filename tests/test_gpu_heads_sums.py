"""The gradients of qk_norm_rope where every sum is exact, so that one (token, head) left out or taken twice shows at any
size; and heads that are not there."""
import pytest
import torch

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


def off_by_one(x):
    """The same values an element off a 16-byte boundary: the scalar kernels."""
    buf = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)
    buf[1:] = x.flatten()
    return buf[1:].view(x.shape)


# tokens, query heads, key heads, head_dim (a power of two), rot_dim, whether the scalar kernels are to take it.  Up to
# 120000 (token, head) terms: each warp walks several items, and each of its lane groups several heads of them.
SIZES = [(5000, 7, 3, 128, 128, False), (20000, 5, 1, 128, 64, False), (3001, 32, 8, 128, 128, False), (2500, 16, 16, 64, 64, False),
         (4001, 9, 2, 256, 256, False), (9000, 3, 1, 32, 32, False), (1500, 2, 2, 512, 512, False), (4000, 9, 4, 128, 128, True),
         (3000, 5, 2, 64, 12, True), (700, 3, 1, 2048, 1024, True)]


@pytest.mark.parametrize("pairs", ["half", "inter"])
@pytest.mark.parametrize("act", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_every_head_counts_once(far, size, act, pairs):
    """Heads of +-1 with eps = 0 and D a power of two: the mean square is 1, exactly, so r is 1 to CUDA's two units in
    the last place, the same for all, and read off the forward pass.  Quarter turns (cosines and sines of 0 and +-1), gradients
    of +-1, +-2, +-3, weights of +-1 and +-2: with r = 1 every product and sum is an integer below 2^24 (a sum over up
    to 120000 terms of 3), or a multiple of 1 / D below 2^13, so the results are exact whatever the order: each head left
    out or taken twice moves every weight's gradient by at least 1.  Padding tokens in between add nothing."""
    tokens, h, hk, d, rot, scalar = size
    g = torch.Generator(device="cuda").manual_seed(tokens + d)
    t = TYPES[act]
    sign = lambda *s: 1.0 - 2.0 * torch.randint(0, 2, s, generator=g, device="cuda").double()  # noqa: E731
    up_to = lambda n, *s: sign(*s) * torch.randint(1, n + 1, s, generator=g, device="cuda").double()  # noqa: E731
    c = torch.tensor([1.0, 0.0, -1.0, 0.0], device="cuda")
    table = torch.cat([c[:, None].expand(4, rot // 2), c.roll(1)[:, None].expand(4, rot // 2)], 1).contiguous()
    pos = torch.randint(0, 4, (tokens,), generator=g, device="cuda")
    pos[torch.randint(0, tokens, (tokens // 50,), generator=g, device="cuda")] = -1
    pos[0] = 0
    live = (pos >= 0)[:, None, None].double()
    place = off_by_one if scalar else (lambda x: x)
    sets = [(sign(tokens, n, d), up_to(3, tokens, n, d), up_to(2, d)) for n in (h, hk)]
    x, dy, w = zip(*[tuple(v.to(t) for v in s) for s in sets])
    x, dy = [place(v) for v in x], [place(v) for v in dy]
    inter = pairs == "inter"
    y, _ = far.qk_norm_rope(x[0].float()[:1], None, torch.ones(d, device="cuda"), None, 0.0, table, pos[:1] * 0, interleaved=inter)
    r = float(y.abs().max())
    assert abs(r - 1.0) <= 2.0 ** -22 and float(y.abs().min()) == r
    got = far.qk_norm_rope_backward(dy[0], dy[1], x[0], x[1], w[0], w[1], 0.0, table, pos, interleaved=inter)
    assert far.device_status() == 0
    cos, sin = c[pos.clamp(min=0)].double()[:, None, None], c.roll(1)[pos.clamp(min=0)].double()[:, None, None]
    for (xd, gd, wd), dx, dw in zip(sets, got[:2], got[2:]):
        a = torch.arange(rot // 2, device="cuda") * (2 if inter else 1)
        b = a + (1 if inter else rot // 2)
        turned = gd.clone()
        turned[..., a], turned[..., b] = gd[..., a] * cos + gd[..., b] * sin, gd[..., b] * cos - gd[..., a] * sin
        want = (live * turned * xd).sum((0, 1))
        hw = turned * wd
        want_dx = live * (hw - xd * (hw * xd).mean(-1, keepdim=True))
        if r == 1.0:
            assert torch.equal(dw.double(), want), f"{int((dw.double() != want).sum())} of {d} sums off"
            assert torch.equal(dx, want_dx.to(t))
        else:  # all terms carry r; a lane's chain, the warps', blocks' and rows' trees: at most 200 additions of 2^-24
            size = r * (live * turned.abs()).sum((0, 1))
            assert bool(((dw.double() - r * want).abs() <= 200 * 2.0 ** -24 * size).all())


@pytest.mark.parametrize("tokens,h,hk,d,scalar", [(8000, 8, 3, 128, False), (30000, 4, 1, 64, False), (8000, 8, 3, 128, True),
                                                  (777, 12, 12, 256, False)])
def test_partial_sums_are_added_without_loss(far, tokens, h, hk, d, scalar):
    """Heads of +-1 again (r = 1), not turned, with gradients of up to 2^14 and the heads' signs: what one block adds up
    (at most 800 heads: below 2^24) is exact, the sum over the blocks is not a binary32 number
    any more, and the weights' gradient is that sum rounded once."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    place = off_by_one if scalar else (lambda x: x)
    table = torch.cat([torch.ones(1, d // 2, device="cuda"), torch.zeros(1, d // 2, device="cuda")], 1).contiguous()
    pos = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    x = [place(1.0 - 2.0 * torch.randint(0, 2, (tokens, n, d), generator=g, device="cuda").float()) for n in (h, hk)]
    dy = [place(v * torch.randint(1, (1 << 14) + 1, v.shape, generator=g, device="cuda").float()) for v in x]
    w = torch.ones(d, device="cuda")
    y, _ = far.qk_norm_rope(x[0][:1].clone(), None, w, None, 0.0, table, pos[:1])
    if not bool((y.abs() == 1.0).all()):
        pytest.skip("r is not 1 here: the terms are not whole numbers")
    got = far.qk_norm_rope_backward(dy[0], dy[1], x[0], x[1], w, w, 0.0, table, pos)
    assert far.device_status() == 0
    for v, gr, dw in zip(x, dy, got[2:]):
        want = (v.double() * gr.double()).sum((0, 1))  # whole numbers below 2^53
        assert float(want.min()) > 2.0 ** 24
        assert torch.equal(dw, want.float()), f"{int((dw != want.float()).sum())} of {d} sums not rounded once"


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_no_query_or_no_key_heads(far, act):
    """A tensor without heads: nothing to normalise, and zeros for its weight's gradient (not what lay in memory)."""
    t, n, d = TYPES[act], 33, 128
    table, pos = far.rope_table(64, d), torch.arange(n, device="cuda")
    w = torch.ones(d, device="cuda", dtype=t)
    some, none = torch.randn(n, 3, d, device="cuda").to(t), torch.empty(n, 0, d, device="cuda", dtype=t)
    alone = far.qk_norm_rope_backward(some, None, some, None, w, None, 1e-6, table, pos)
    for q, k, filled in ((some, none, 0), (none, some, 1), (none, none, None)):
        y = far.qk_norm_rope(q, k, w, w, 1e-6, table, pos)
        assert y[0].shape == q.shape and y[1].shape == k.shape
        used = [torch.full((d,), float("nan"), device="cuda") for _ in range(64)]
        torch.cuda.synchronize()
        del used  # what the allocator hands out next holds NaN
        got = far.qk_norm_rope_backward(q, k, q, k, w, w, 1e-6, table, pos)
        assert far.device_status() == 0
        for i in (0, 1):
            if i == filled:
                assert torch.equal(got[2 + i], alone[2]) and torch.equal(got[i], alone[0])
            else:
                assert bool((got[2 + i] == 0).all()) and got[i].numel() == 0
