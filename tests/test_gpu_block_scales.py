"""gemm_fp8_block with scales from all of binary32's range, infinite and NaN ones among them, on every kernel: few rows
of x (16, 32 and 64 a CTA), CTA pairs, and the plain kernel, with wt scaled by tiles and by rows.

The reference takes the definition block by block in 64 bits: term = xs * ws * (sum over the block of x * w).  A sum
lies between 2^-18 and 2^25 or is 0, so a term is a binary32 number, to a few units of 2^-24, wherever it lies in
binary32's range at all, although xs * ws or a sum times one of its scales may leave that range on the way."""
import pytest
import torch

from block_ref import BLOCK, nblocks
from heads_ref import SMALLEST, half_step

pytestmark = pytest.mark.gpu
TOP = torch.finfo(torch.float32).max


@pytest.fixture(scope="module")
def far():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import mixed_precision_residual_gb300 as far

    return far


# rows of x, k, how wt is scaled, the kernel: (kind, rows of x a CTA) of far_plan_gemm_fp8_for_sms
N = 392
KERNELS = [(3, 512, "tile", (2, 16)), (3, 512, "row", (2, 16)), (20, 512, "tile", (2, 32)), (20, 512, "row", (2, 32)),
           (200, 512, "row", (2, 64)), (700, 512, "tile", (1, 0)), (200, 128, "tile", (1, 0)), (200, 128, "row", (1, 0)),
           (3000, 512, "row", (1, 0)), (70, 520, "tile", (0, 0)), (70, 520, "row", (0, 0))]


def codes(g, rows, k, small=False):
    """E4M3 codes without NaN; small: the seven values next to zero, of either sign."""
    c = torch.randint(0, 8 if small else 127, (rows, k), generator=g, device="cuda", dtype=torch.int32)
    return (c + 128 * torch.randint(0, 2, (rows, k), generator=g, device="cuda", dtype=torch.int32)).to(torch.uint8)


def terms(xq, xs, wq, ws):
    """[blocks, m, n] in 64 bits: the scaled sum of each block, and the same of the magnitudes."""
    value = lambda c: c.view(torch.float8_e4m3fn).double()  # noqa: E731
    w_scale = ws.double() if ws.shape[0] == wq.shape[0] else ws.double().repeat_interleave(BLOCK, 0)[:wq.shape[0]]
    out, size = [], []
    for b in range(nblocks(xq.shape[1])):
        x, w = value(xq[:, b * BLOCK:(b + 1) * BLOCK]), value(wq[:, b * BLOCK:(b + 1) * BLOCK])
        f = xs[:, b].double()[:, None] * w_scale[:, b].double()[None, :]
        out.append(f * (x @ w.T))
        size.append(f.abs() * (x.abs() @ w.abs().T))
    return torch.stack(out), torch.stack(size)


def check(far, kernel, xq, xs, wq, ws, dtype=torch.float32, where=""):
    """Every output whose terms all lie in range within the bound of its binary32 steps (block_ref.product's, and one
    rounding a term and a sum to binary32's smallest step); one with one term past the range infinite, of its sign;
    infinite and NaN scales as the definition has them."""
    (m, k), n = xq.shape, wq.shape[0]
    plan = far.plan_gemm_fp8_for_sms(m, n, k, "row" if ws.shape[0] == n else "tile",
                                     torch.cuda.get_device_properties(0).multi_processor_count)
    assert (plan["kind"], plan["rows"]) == kernel, "the shape no longer reaches the kernel it is meant for"
    y = far.gemm_fp8_block(xq, xs, wq, ws, out_dtype=dtype).double()
    assert far.device_status() == 0
    t, size = terms(xq, xs, wq, ws)
    ref, total = t.sum(0), size.sum(0)
    fine = total < TOP / 2
    err = (min(k, BLOCK) + len(t) + 4) * 2.0 ** -22 * total + 2 * len(t) * 2.0 ** -150
    allowed = err + half_step(dtype) * (ref.abs() + err) + SMALLEST[dtype]
    bad = fine & ~((y - ref).abs() <= allowed)
    assert not bad.any(), (f"{where}: {int(bad.sum())} of {int(fine.sum())} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{float(y[bad][0])} for {float(ref[bad][0])}")
    past = (t.abs() > 1.01 * TOP) & ~t.isinf()
    rest = torch.where(past, 0.0, size).sum(0) < TOP / 4
    one = (past.sum(0) == 1) & rest
    want = torch.sign(torch.where(past, t, 0.0).sum(0)) * float("inf")
    assert torch.equal(y[one], want[one]), f"{where}: a term past the range"
    special = (~t.isfinite()).any(0) & ~past.any(0) & (torch.where(t.isfinite(), size, 0.0).sum(0) < TOP / 2)
    assert torch.equal(y[special].isnan(), ref[special].isnan()), f"{where}: NaN"
    inf = special & ref.isinf()
    assert torch.equal(y[inf], ref[inf]), f"{where}: infinities"
    return fine, one, special


# powers of two of x's and wt's scales: their product below binary32's smallest normal number and above its largest one,
# a sum times the first or the second scale out of range on the way, denormal scales
PAIRS = [(-80, -70), (-70, -60), (-63, -64), (-100, -40), (-40, -100), (-149, 20), (20, -149), (-126, 22), (22, -126), (70, -70),
         (110, -100), (-100, 110), (126, -126), (-126, 126), (127, -149), (-149, 127), (60, 40), (40, 60)]


@pytest.mark.parametrize("m,k,rows,kernel", KERNELS, ids=str)
def test_scales_of_every_size(far, m, k, rows, kernel):
    g = torch.Generator(device="cuda").manual_seed(m + k)
    xq, wq = codes(g, m, k), codes(g, N, k)
    kb, wn = nblocks(k), N if rows == "row" else nblocks(N)
    one_to_two = lambda r: 1 + torch.rand(r, kb, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    for a, b in PAIRS:
        xs, ws = (one_to_two(m) * 2.0 ** a).float(), (one_to_two(wn) * 2.0 ** b).float()
        fine, _, _ = check(far, kernel, xq, xs, wq, ws, where=f"2^{a}, 2^{b}")
        assert bool(fine.all())
        # a row and a column (or a tile's) of zero scales beside them: zeros
        xs[1], ws[1] = 0.0, 0.0
        check(far, kernel, xq, xs, wq, ws, dtype=torch.bfloat16, where=f"2^{a}, 2^{b} and zeros")
    xs, ws = torch.full((m, kb), 3.0e38, device="cuda"), torch.zeros(wn, kb, device="cuda")
    assert bool((far.gemm_fp8_block(xq, xs, wq, ws, out_dtype=torch.float32) == 0).all()), "zero scales beside large ones"


@pytest.mark.parametrize("m,k,rows,kernel", KERNELS, ids=str)
def test_products_past_the_range_of_small_sums(far, m, k, rows, kernel):
    """xs * ws is past binary32's largest number, the sums are so small that the terms are not; zero sums give zeros."""
    g = torch.Generator(device="cuda").manual_seed(m + k + 1)
    xq, wq = codes(g, m, k, small=True), codes(g, N, k, small=True)
    xq[0] = 0
    wq[3] = 0
    kb, wn = nblocks(k), N if rows == "row" else nblocks(N)
    xs, ws = torch.full((m, kb), 2.0 ** 68, device="cuda"), torch.full((wn, kb), 2.0 ** 62, device="cuda")
    fine, _, _ = check(far, kernel, xq, xs, wq, ws)
    assert bool(fine.all())
    y = far.gemm_fp8_block(xq, xs, wq, ws, out_dtype=torch.float32)
    assert bool((y[0] == 0).all()) and bool((y[:, 3] == 0).all()) and bool((y != 0).any())


@pytest.mark.parametrize("m,k,rows,kernel", KERNELS, ids=str)
def test_mixed_scales(far, m, k, rows, kernel):
    """Rows and columns of every size side by side, from block to block another: ordinary ones must not suffer."""
    g = torch.Generator(device="cuda").manual_seed(m + k + 2)
    xq, wq = codes(g, m, k), codes(g, N, k)
    kb, wn = nblocks(k), N if rows == "row" else nblocks(N)
    pick = torch.tensor([-149.0, -120.0, -60.0, 0.0, 0.0, 0.0, 0.0, 50.0, 101.0, 126.0], dtype=torch.float64, device="cuda")
    size = lambda r: (torch.exp2(pick[torch.randint(0, len(pick), (r, kb), generator=g, device="cuda")]) *  # noqa: E731
                      (1 + torch.rand(r, kb, generator=g, device="cuda"))).float()
    for _ in range(6):
        fine, one, _ = check(far, kernel, xq, size(m), wq, size(wn))
        assert float(fine.float().mean()) > 0.05  # (half of them on average; a row of large scales has few, and there may be 3 rows)


@pytest.mark.parametrize("m,k,rows,kernel", KERNELS, ids=str)
def test_infinite_and_nan_scales_and_codes(far, m, k, rows, kernel):
    g = torch.Generator(device="cuda").manual_seed(m + k + 3)
    xq, wq = codes(g, m, k), codes(g, N, k)
    kb, wn = nblocks(k), N if rows == "row" else nblocks(N)
    inf, nan, last = float("inf"), float("nan"), kb - 1
    xs, ws = torch.rand(m, kb, generator=g, device="cuda") + 0.5, torch.rand(wn, kb, generator=g, device="cuda") + 0.5
    fine, _, special = check(far, kernel, xq, xs, wq, ws)
    assert bool(fine.all()) and not bool(special.any())
    xs[0, 0], xs[1, last], xs[2, 0] = inf, nan, -inf
    ws[1, last] = inf  # meets xs[2]'s infinity in another block, or the same one (one block of k)
    _, _, special = check(far, kernel, xq, xs, wq, ws, where="infinite scales")
    assert bool(special[:3].all())
    ws[2, 0] = nan
    _, _, special = check(far, kernel, xq, xs, wq, ws, where="NaN scales")
    assert float(special.float().mean()) > (0.002 if rows == "row" else 0.1)
    ws[2, 0] = 0.0  # zero beside an infinity: NaN by the definition
    check(far, kernel, xq, xs, wq, ws, where="zero beside infinity")
    xs, ws = torch.rand(m, kb, generator=g, device="cuda") + 0.5, torch.rand(wn, kb, generator=g, device="cuda") + 0.5
    xq[1, 5], wq[300, k - 3] = 0x7F, 0xFF
    xs[2], ws[0] = 3.0e38, 3.0e38
    _, _, special = check(far, kernel, xq, xs, wq, ws, where="NaN codes")
    nans = torch.zeros(m, N, dtype=torch.bool, device="cuda")
    nans[1], nans[:, 300] = True, True
    assert torch.equal(far.gemm_fp8_block(xq[:, :], xs / xs, wq, ws / ws, out_dtype=torch.float32).isnan(), nans)


@pytest.mark.parametrize("m,k,rows,kernel", KERNELS, ids=str)
def test_far_scales_that_do_not_meet(far, m, k, rows, kernel):
    """Tiny scales of x in some blocks and of wt in others, no product of two out of range: the results of ordinary
    scales times the powers of two, bit for bit where every block's scales are the same power of two apart."""
    g = torch.Generator(device="cuda").manual_seed(m + k + 4)
    xq, wq = codes(g, m, k), codes(g, N, k)
    kb, wn = nblocks(k), N if rows == "row" else nblocks(N)
    xs, ws = torch.rand(m, kb, generator=g, device="cuda") + 0.5, torch.rand(wn, kb, generator=g, device="cuda") + 0.5
    want = far.gemm_fp8_block(xq, xs, wq, ws, out_dtype=torch.float32)
    a = torch.tensor([-90.0 if b % 2 else -10.0 for b in range(kb)], device="cuda")
    far_x, far_w = xs * torch.exp2(a), ws * torch.exp2(-100.0 - a)  # block by block a product 2^-100 of the one before
    check(far, kernel, xq, far_x, wq, far_w)
    got = far.gemm_fp8_block(xq, far_x, wq, far_w, out_dtype=torch.float32)
    assert torch.equal(got, want * 2.0 ** -100)


@pytest.mark.parametrize("dtype,columns", [(torch.float32, 2056), (torch.bfloat16, 2050)])
@pytest.mark.parametrize("rows", ["tile", "row"])
def test_second_pass_over_several_tiles(far, rows, dtype, columns):
    """Far scales in a few places of a product of three tiles a CTA pair: all of it is right, with outputs that leave by TMA
    and with ones that are stored row by row (rows off a 16-byte boundary)."""
    m, k = 5200, 656
    g = torch.Generator(device="cuda").manual_seed(columns)
    xq, wq = codes(g, m, k), codes(g, columns, k)
    kb, wn = nblocks(k), columns if rows == "row" else nblocks(columns)
    xs, ws = torch.rand(m, kb, generator=g, device="cuda") + 0.5, torch.rand(wn, kb, generator=g, device="cuda") + 0.5
    usual = far.gemm_fp8_block(xq, xs, wq, ws, out_dtype=dtype)
    xs[[3, 2600, m - 1], [0, 3, kb - 1]] = torch.tensor([2.0 ** -120, 2.0 ** 100, 0.0], device="cuda")
    ws[[0, wn // 2, wn - 1], [0, 3, kb - 1]] = torch.tensor([2.0 ** -20, 2.0 ** -110, 2.0 ** 105], device="cuda")
    check(far, (1, 0), xq, xs, wq, ws, dtype=dtype, where=rows)
    again = far.gemm_fp8_block(xq, xs, wq, ws, out_dtype=dtype)
    assert torch.equal(far.gemm_fp8_block(xq, xs, wq, ws, out_dtype=dtype), again)
    same = torch.ones(m, columns, dtype=torch.bool, device="cuda")
    same[[3, 2600, m - 1]] = False
    cols = torch.arange(columns, device="cuda") // (1 if rows == "row" else BLOCK)
    for j in (0, wn // 2, wn - 1):
        same[:, cols == j] = False
    # Elsewhere the scales are the usual ones, and the tensor cores' sums the same bits in either pass: a term is rounded
    # twice and added once, each of it by at most 2^-24 of the terms' magnitudes T that have been added, so each
    # result is within 3 * blocks * 2^-24 T of the exact sum of those terms, and rounded once to dtype.
    _, size = terms(xq, xs, wq, ws)
    bound = 2 * 3 * kb * 2.0 ** -24 * size.sum(0)[same]
    off = (again[same].double() - usual[same].double()).abs()
    assert bool((off <= bound + torch.finfo(dtype).eps * (usual[same].double().abs() + bound)).all())
