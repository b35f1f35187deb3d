"""GPU parity of the dense 8-bit product, the grouped products and the grouped
weight gradient with the float64 definitions.

Tolerance: |c - ref| <= rel * sum of magnitudes + one spacing of the output
type.  The tensor core adds 16 (16-bit) or 32 (8-bit) products a step into an
fp32 accumulator, losing at most 2^-22 of the running magnitude a step
(truncation, and the alignment of the step's terms); the 8-bit product also
adds one fp32 term per block of 128, two roundings each.  So rel =
(steps + 8) * 2^-22 with steps the MMA steps along K (16-bit) or 4 + the number
of blocks (8-bit).
"""

import numpy as np
import pytest

from oracle import operators as OO
from oracle import tolerance as OT

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402
from tile_size_decision_gb300 import _abi  # noqa: E402

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ws():
    T.load()
    return T.workspace()


def f64(t):
    return t.double().cpu().numpy()


def draw(shape, dtype, seed, scale=1.0, pitch=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    *lead, cols = shape
    t = torch.randn((*lead, pitch or (cols + 7) // 8 * 8), generator=g, device="cuda") * scale
    return t.to(DT[dtype])[..., :cols]


def rel16(k):
    return ((k + 15) // 16 + 8) * 2.0 ** -22


def rel8(k):
    return (4 + OO.blocks(k) + 8) * 2.0 ** -22


def assert_close(got, ref, bound, dtype, rel):
    ok, worst, idx = OT.check(f64(got), ref, bound, dtype, rel)
    assert ok, f"worst error/tolerance {worst} at {idx}"


def offsets_of(sizes, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(sizes)]), dtype=torch.int32,
                        device="cuda")


# ---- dense 8-bit product -------------------------------------------------------------

DENSE = [(1, 1, 1), (1, 16, 16), (1, 128, 128), (7, 100, 48), (16, 512, 1024), (17, 129, 640),
         (33, 130, 272), (64, 256, 4096), (65, 300, 400), (130, 257, 400), (300, 520, 1000),
         (257, 1024, 2050), (1000, 768, 512), (2, 4096, 8192), (1024, 2048, 384)]


def fp8_operands(m, n, k, seed, spread=True):
    a, b = draw((m, k), "f32", seed), draw((n, k), "f32", seed + 1)
    if spread:                       # rows and blocks of very different sizes
        a = a * torch.exp2(torch.arange(m, device="cuda") % 13 - 6.0)[:, None]
    a8, sa = T.quantize_fp8(a.contiguous())
    b8, sb = T.quantize_fp8(b.contiguous(), block_rows=128)
    return a8, sa, b8, sb


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", DENSE, ids=str)
def test_dense_8bit(ws, shape, out):
    m, n, k = shape
    a8, sa, b8, sb = fp8_operands(m, n, k, 7)
    c = T.gemm_fp8(a8, sa, b8, sb, out_dtype=out, workspace=ws)
    T.check(ws)
    ref, bound = OO.gemm_fp8(f64(a8), f64(sa), f64(b8), f64(sb))
    assert_close(c, ref, bound, out, rel8(k))
    # Either order of the row scales, and a product that runs again, give the same bits.
    again = T.gemm_fp8(a8, sa.contiguous(), b8, sb.t().contiguous().t(), out_dtype=out, workspace=ws)
    T.check(ws)
    assert torch.equal(again, c)


@pytest.mark.parametrize("shape", [(20, 130, 272), (300, 520, 640)], ids=str)
def test_dense_8bit_writes_only_its_rows_and_columns(ws, shape):
    m, n, k = shape
    a8, sa, b8, sb = fp8_operands(m, n, k, 9)
    full = torch.full((m + 2, n + 9), 5.0, dtype=torch.float32, device="cuda")
    T.gemm_fp8(a8, sa, b8, sb, out=full[1:m + 1, 3:n + 3], workspace=ws)
    T.check(ws)
    ref, bound = OO.gemm_fp8(f64(a8), f64(sa), f64(b8), f64(sb))
    assert_close(full[1:m + 1, 3:n + 3], ref, bound, "f32", rel8(k))
    full[1:m + 1, 3:n + 3] = 5.0
    assert bool((full == 5.0).all())


@pytest.mark.parametrize("m", [5, 200])
def test_dense_8bit_keeps_a_nan_in_its_row(ws, m):
    a8, sa, b8, sb = fp8_operands(m, 130, 256, 11)
    sa = sa.clone()
    sa[3, 1] = float("nan")
    c = T.gemm_fp8(a8, sa, b8, sb, out_dtype="f32", workspace=ws)
    T.check(ws)
    assert bool(c[3].isnan().all())
    assert int(c.isnan().any(1).sum()) == 1


def test_dense_8bit_of_no_rows_and_of_another_stream(ws):
    a8, sa, b8, sb = fp8_operands(128, 512, 512, 13)
    assert T.gemm_fp8(a8[:0], sa[:0], b8, sb, workspace=ws).shape == (0, 512)
    want = T.gemm_fp8(a8, sa, b8, sb, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = T.gemm_fp8(a8, sa, b8, sb, workspace=ws, stream=side)
    side.synchronize()
    T.check(ws)
    assert torch.equal(got, want)


# ---- grouped products ------------------------------------------------------------------

SIZES = {
    "one": [5],
    "few": [1, 0, 3, 2, 0, 1],
    "edges": [15, 16, 17, 0, 31, 33, 64, 1],
    "tiles": [127, 128, 129, 0, 257, 1, 255],
    "skewed": [700, 0, 0, 3],
    "many": [i % 5 for i in range(70)],
    "none": [0, 0, 0],
}


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f16")])
@pytest.mark.parametrize("nk", [(64, 64), (130, 72), (1, 8), (520, 1000), (257, 264)], ids=str)
@pytest.mark.parametrize("trans_b", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("sizes", list(SIZES), ids=str)
def test_grouped_16bit(ws, sizes, trans_b, nk, dtype, out):
    n, k = nk
    groups = SIZES[sizes]
    t = sum(groups)
    off = offsets_of(groups)
    a = draw((t, k), dtype, 60)
    w = draw((len(groups), n, k) if trans_b else (len(groups), k, n), dtype, 61)
    c = T.grouped_gemm(a, w, off, trans_b=trans_b, out_dtype=out, workspace=ws)
    T.check(ws)
    ref, bound = OO.grouped(f64(a), f64(w), off.tolist(), trans_b)
    assert_close(c, ref, bound, out, rel16(k))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("nk", [(64, 64), (130, 72), (520, 1000), (257, 2064)], ids=str)
@pytest.mark.parametrize("sizes", list(SIZES), ids=str)
def test_grouped_8bit(ws, sizes, nk, out):
    n, k = nk
    groups = SIZES[sizes]
    t = sum(groups)
    off = offsets_of(groups)
    a8, sa = T.quantize_fp8(draw((t, k), "f32", 62))
    b8, sb = T.quantize_fp8(draw((len(groups), n, k), "f32", 63), block_rows=128)
    c = T.grouped_gemm_fp8(a8, sa, b8, sb, off, out_dtype=out, workspace=ws)
    T.check(ws)
    ref, bound = OO.grouped_fp8(f64(a8), f64(sa), f64(b8), f64(sb), off.tolist())
    assert_close(c, ref, bound, out, rel8(k))


@pytest.mark.parametrize("sizes", [[3, 0, 20], [130, 300, 70]], ids=str)
def test_grouped_rows_outside_every_group_stay_untouched(ws, sizes):
    n, k = 200, 136
    off = offsets_of(sizes, first=4)
    t = sum(sizes) + 9
    a, w = draw((t, k), "bf16", 64), draw((len(sizes), k, n), "bf16", 65)
    full = torch.full((t, n + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    T.grouped_gemm(a, w, off, out=full[:, 4:n + 4], workspace=ws)
    T.check(ws)
    ref, bound = OO.grouped(f64(a), f64(w), off.tolist())
    inside = slice(4, 4 + sum(sizes))
    assert_close(full[inside, 4:n + 4], ref[inside], bound[inside], "bf16", rel16(k))
    full[inside, 4:n + 4] = 3.0
    assert bool((full == 3.0).all())


@pytest.mark.parametrize("sizes", [[5, 7], [130, 140]], ids=str)
def test_grouped_nan_of_one_group_stays_in_it(ws, sizes):
    n, k = 136, 200
    off = offsets_of(sizes)
    a, w = draw((sum(sizes), k), "f16", 66), draw((2, k, n), "f16", 67)
    dc = draw((sum(sizes), n), "f16", 68)
    a[sizes[0]:] = float("nan")
    dc[sizes[0]:] = float("inf")
    c = T.grouped_gemm(a, w, off, workspace=ws)
    dw = T.grouped_wgrad(a, dc, off, workspace=ws)
    T.check(ws)
    assert not bool(c[:sizes[0]].isnan().any()) and bool(c[sizes[0]:].isnan().all())
    assert bool(dw[0].isfinite().all()) and bool(dw[1].isnan().all())
    ref, bound = OO.wgrad(f64(a), f64(dc), off.tolist())
    assert_close(dw[0], ref[0], bound[0], "f16", rel16(sizes[0]))


def test_grouped_offsets_out_of_range_stay_in_bounds(ws):
    # Offsets below zero, past the rows and descending count as the nearer
    # end and as empty groups.
    a, w = draw((40, 64), "bf16", 69), draw((3, 64, 128), "bf16", 70)
    off = torch.tensor([-5, 12, 10, 90], dtype=torch.int32, device="cuda")
    c = torch.zeros((40, 128), dtype=torch.float32, device="cuda")
    T.grouped_gemm(a, w, off, out=c, workspace=ws)
    dw = T.grouped_wgrad(a, a, off, out_dtype="f32", workspace=ws)
    T.check(ws)
    ref0, b0 = OO.grouped(f64(a[:10]), f64(w[:1]), [0, 10])
    ref2, b2 = OO.grouped(f64(a[12:]), f64(w[2:]), [0, 28])
    assert_close(c[:10], ref0, b0, "f32", rel16(64))
    assert_close(c[12:], ref2, b2, "f32", rel16(64))
    assert bool((dw[1] == 0).all())


def test_grouped_strides_and_the_largest_group_count(ws):
    groups, n, k = 4096, 24, 16
    sizes = np.zeros(groups, dtype=int)
    sizes[[0, 31, 32, 1000, 4095]] = [3, 1, 40, 2, 5]
    off = offsets_of(sizes)
    a = draw((int(sizes.sum()), k), "bf16", 71, pitch=40)
    w = draw((groups, k, n), "bf16", 72, pitch=32)
    c = T.grouped_gemm(a, w, off, out_dtype="f32", workspace=ws)
    T.check(ws)
    ref, bound = OO.grouped(f64(a), f64(w), off.tolist())
    assert_close(c, ref, bound, "f32", rel16(k))


def test_grouped_repeat_is_deterministic(ws):
    off = offsets_of([3, 0, 9, 2])
    a, w = draw((14, 2048), "bf16", 73), draw((4, 2048, 256), "bf16", 74)
    first = T.grouped_gemm(a, w, off, workspace=ws)
    for _ in range(3):
        assert torch.equal(T.grouped_gemm(a, w, off, workspace=ws), first)
    T.check(ws)


# ---- weight gradients ---------------------------------------------------------------------


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("kn", [(64, 64), (72, 136), (8, 8), (200, 520), (264, 257), (129, 1)], ids=str)
@pytest.mark.parametrize("sizes", list(SIZES), ids=str)
def test_wgrad(ws, sizes, kn, dtype, out):
    k, n = kn
    groups = SIZES[sizes]
    t = sum(groups)
    off = offsets_of(groups)
    a, dc = draw((t, k), dtype, 80), draw((t, n), dtype, 81)
    full = torch.full((len(groups), k + 1, n + 3), 9.0, dtype=DT[out], device="cuda")
    T.grouped_wgrad(a, dc, off, out=full[:, :k, :n], workspace=ws)
    T.check(ws)
    ref, bound = OO.wgrad(f64(a), f64(dc), off.tolist())
    assert_close(full[:, :k, :n], ref, bound, out, rel16(max(groups)))
    full[:, :k, :n] = 9.0
    assert bool((full == 9.0).all())
    dw = T.grouped_wgrad(a, dc, off, out_dtype=out, workspace=ws)
    T.check(ws)
    assert_close(dw, ref, bound, out, rel16(max(groups)))


def test_gradients_against_differences(ws):
    # The product is linear in the rows and in the weight: for steps and
    # operands that are small integers every difference is exact.
    sizes = [3, 0, 5]
    off = offsets_of(sizes)
    g = torch.Generator(device="cuda").manual_seed(90)

    def ints(*shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").to(torch.bfloat16)

    a, w, dc = ints(8, 32), ints(3, 32, 40), ints(8, 40)
    da = T.grouped_gemm(dc, w, off, trans_b=True, out_dtype="f32", workspace=ws)
    dw = T.grouped_wgrad(a, dc, off, out_dtype="f32", workspace=ws)

    def loss(a_, w_):
        c = T.grouped_gemm(a_, w_, off, out_dtype="f32", workspace=ws)
        return float((c * dc.float()).sum())

    base = loss(a, w)
    for i, j in [(0, 0), (2, 31), (7, 5)]:
        s = torch.zeros_like(a)
        s[i, j] = 1
        assert loss(a + s, w) - base == float(da[i, j])
    for e, i, j in [(0, 0, 0), (1, 4, 4), (2, 31, 39)]:
        s = torch.zeros_like(w)
        s[e, i, j] = 1
        assert loss(a, w + s) - base == float(dw[e, i, j])
    T.check(ws)


# ---- waits and refusals ----------------------------------------------------------------------


def expect_timeout(ws):
    with pytest.raises(T.TilesError) as e:
        T.check(ws)
    assert e.value.status == _abi.ERR_TIMEOUT
    T.check(ws)


@pytest.mark.parametrize("rows", [20, 600])
@pytest.mark.parametrize("kind", ["fp8", "grouped", "dgrad", "wgrad"])
def test_product_wait_expires_and_the_context_recovers(ws, kind, rows):
    k = n = 512
    off = offsets_of([rows])
    a, w = draw((rows, k), "bf16", 91), draw((1, k, n), "bf16", 92)
    a8, sa = T.quantize_fp8(a)
    b8, sb = T.quantize_fp8(w[0].t().contiguous(), block_rows=128)

    def call():
        if kind == "fp8":
            return T.gemm_fp8(a8, sa, b8, sb, workspace=ws)
        if kind == "wgrad":
            return T.grouped_wgrad(a, a, off, workspace=ws)
        return T.grouped_gemm(a, w, off, trans_b=kind == "dgrad", workspace=ws)

    want = call()
    T.check(ws)
    T.selftest_drop_stage(0, 50_000_000)
    call()
    expect_timeout(ws)
    got = call()
    T.check(ws)
    assert torch.equal(got, want)


def test_python_refusals(ws):
    a8, sa, b8, sb = fp8_operands(4, 128, 128, 95)
    with pytest.raises(TypeError):
        T.gemm_fp8(a8.float(), sa, b8, sb, workspace=ws)
    with pytest.raises(ValueError):
        T.gemm_fp8(a8, sa[:3], b8, sb, workspace=ws)
    with pytest.raises(ValueError):
        T.gemm_fp8(a8, sa, b8[:, :64], sb, workspace=ws)
    with pytest.raises(T.TilesError):
        T.gemm_fp8(a8, sa, b8, sb)
    a, w = draw((4, 64), "bf16", 96), draw((2, 64, 64), "bf16", 97)
    off = offsets_of([2, 2])
    with pytest.raises(ValueError):
        T.grouped_gemm(a, w, off.long(), workspace=ws)
    with pytest.raises(ValueError):
        T.grouped_gemm(a, w, off[:2], workspace=ws)
    with pytest.raises(TypeError):
        T.grouped_gemm(a.half(), w, off, workspace=ws)
    with pytest.raises(T.TilesError):
        T.grouped_gemm(draw((4, 64), "bf16", 98, pitch=66), w, off, workspace=ws)
    with pytest.raises(ValueError):
        T.grouped_wgrad(a, a[:3], off, workspace=ws)


# ---- sizes that take the large tiles -----------------------------------------------------
# (Enough rows that the large-tile kernels are chosen; the float64 products are
# made on the device.)


def dev_fp8(a8, sa, b8, sb):
    """(product, sum of magnitudes) of one weight in float64, on the device."""
    ref = torch.zeros((a8.shape[0], b8.shape[0]), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(ref)
    for t in range(sa.shape[1]):
        part = slice(128 * t, min(128 * (t + 1), a8.shape[1]))
        s = sa[:, t].double()[:, None] * sb[:, t].double().repeat_interleave(128)[: b8.shape[0]]
        x, w = a8[:, part].double(), b8[:, part].double()
        ref += s * (x @ w.t())
        bound += s.abs() * (x.abs() @ w.abs().t())
    return ref, bound


def dev_grouped(a, w, off, trans_b):
    n = w.shape[1] if trans_b else w.shape[2]
    ref = torch.zeros((a.shape[0], n), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(ref)
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        x, b = a[lo:hi].double(), (w[e].t() if trans_b else w[e]).double()
        ref[lo:hi], bound[lo:hi] = x @ b, x.abs() @ b.abs()
    return ref, bound


def assert_close_dev(got, ref, bound, dtype, rel):
    assert_close(got, f64(ref), f64(bound), dtype, rel)


LARGE_DENSE = [(3000, 2050, 1040), (20000, 130, 528), (1100, 4100, 2064), (2100, 4100, 1040),
               (1100, 1030, 2064)]


@pytest.mark.parametrize("out,shift", [("bf16", 0), ("f16", 0), ("f32", 0), ("f32", 3), ("bf16", 1)])
@pytest.mark.parametrize("shape", LARGE_DENSE, ids=str)
def test_dense_8bit_large_tiles(ws, shape, out, shift):
    # `shift`: the result starts off a 16-byte boundary (it cannot leave in boxes).
    m, n, k = shape
    a8, sa, b8, sb = fp8_operands(m, n, k, 17)
    sa = sa.clone()
    sa[m - 2, 1] = float("nan")
    full = torch.full((m + 2, (n + 23) // 8 * 8), 5.0, dtype=DT[out], device="cuda")
    got = full[1:m + 1, shift:n + shift]
    T.gemm_fp8(a8, sa, b8, sb, out=got, workspace=ws)
    T.check(ws)
    rows = torch.cat([torch.arange(0, 520), torch.arange(m - 300, m)]).cuda()
    assert bool(got[m - 2].isnan().all()) and int(got.isnan().any(1).sum()) == 1
    keep = rows[rows != m - 2]
    ref, bound = dev_fp8(a8[keep], sa[keep], b8, sb)
    assert_close_dev(got[keep], ref, bound, out, rel8(k))
    again = torch.empty((m, n), dtype=DT[out], device="cuda")
    T.gemm_fp8(a8, sa, b8, sb, out=again, workspace=ws)
    T.check(ws)
    assert torch.equal(again[: m - 2], got[: m - 2])
    got.fill_(5.0)
    assert bool((full == 5.0).all())


LARGE_GROUPS = {
    "heavy": ([900, 1300, 0, 2100, 800], 1500, 1040),
    "ragged": ([700, 0, 257, 1, 300, 2000], 1003, 1000),
    "wide": ([1, 5200, 256, 0, 255, 3], 600, 1040),
    "many": ([300 * (i % 3) for i in range(70)], 264, 1032),
    "uneven": ([0, 2500, 0], 1100, 264),
}


@pytest.mark.parametrize("dtype,out,shift", [("bf16", "bf16", 0), ("f16", "f32", 0),
                                             ("bf16", "f32", 1), ("f16", "f16", 5)])
@pytest.mark.parametrize("trans_b", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("name", list(LARGE_GROUPS))
def test_grouped_16bit_large_tiles(ws, name, trans_b, dtype, out, shift):
    sizes, n, k = LARGE_GROUPS[name]
    off = offsets_of(sizes, first=2)
    t = sum(sizes) + 5
    a = draw((t, k), dtype, 101)
    w = draw((len(sizes), n, k) if trans_b else (len(sizes), k, n), dtype, 102)
    # The rows outside every group, and the group after the first, are not numbers.
    a[:2] = a[t - 3:] = float("nan")
    bad = slice(2 + sizes[0], 2 + sizes[0] + sizes[1])
    a[bad] = float("inf")
    full = torch.full((t, (n + 23) // 8 * 8), 5.0, dtype=DT[out], device="cuda")
    got = full[:, shift:n + shift]
    T.grouped_gemm(a, w, off, trans_b=trans_b, out=got, workspace=ws)
    T.check(ws)
    assert not bool(got[bad].isfinite().any())
    a[bad] = 0
    got[bad] = 0
    ref, bound = dev_grouped(a, w, off.tolist(), trans_b)
    inside = slice(2, t - 3)
    assert_close_dev(got[inside], ref[inside], bound[inside], out, rel16(k))
    got[inside] = 5.0
    assert bool((full == 5.0).all())


@pytest.mark.parametrize("out,shift", [("bf16", 0), ("f32", 0), ("f32", 2)])
@pytest.mark.parametrize("name", list(LARGE_GROUPS))
def test_grouped_8bit_large_tiles(ws, name, out, shift):
    sizes, n, k = LARGE_GROUPS[name]
    off = offsets_of(sizes, first=1)
    t = sum(sizes) + 3
    a8, sa = T.quantize_fp8(draw((t, k), "f32", 103))
    b8, sb = T.quantize_fp8(draw((len(sizes), n, k), "f32", 104), block_rows=128)
    sa = sa.clone()
    sa[0] = sa[t - 2:] = float("nan")
    full = torch.full((t, (n + 23) // 8 * 8), 5.0, dtype=DT[out], device="cuda")
    got = full[:, shift:n + shift]
    T.grouped_gemm_fp8(a8, sa, b8, sb, off, out=got, workspace=ws)
    T.check(ws)
    for e, (lo, hi) in enumerate(zip(off.tolist()[:-1], off.tolist()[1:])):
        if hi > lo:
            ref, bound = dev_fp8(a8[lo:hi], sa[lo:hi], b8[e], sb[e])
            assert_close_dev(got[lo:hi], ref, bound, out, rel8(k))
    got[1:t - 2] = 5.0
    assert bool((full == 5.0).all())


@pytest.mark.parametrize("kind", ["fp8", "grouped", "dgrad", "grouped_fp8"])
def test_large_tile_wait_expires_and_the_context_recovers(ws, kind):
    rows, k, n = 2500, 1024, 1104
    off = offsets_of([rows - 300, 300])
    a, w = draw((rows, k), "bf16", 105), draw((2, k, n), "bf16", 106)
    wt = w.transpose(1, 2).contiguous()
    a8, sa = T.quantize_fp8(a)
    b8, sb = T.quantize_fp8(wt, block_rows=128)

    def call():
        if kind == "fp8":
            return T.gemm_fp8(a8, sa, b8[0], sb[0], workspace=ws)
        if kind == "grouped_fp8":
            return T.grouped_gemm_fp8(a8, sa, b8, sb, off, workspace=ws)
        return T.grouped_gemm(a, wt if kind == "dgrad" else w, off, trans_b=kind == "dgrad",
                              workspace=ws)

    want = call()
    T.check(ws)
    for stage in (0, 2):
        T.selftest_drop_stage(stage, 50_000_000)
        call()
        expect_timeout(ws)
        got = call()
        T.check(ws)
        assert torch.equal(got, want)


@pytest.mark.parametrize("kn", [(264, 257), (200, 518), (40, 4)], ids=str)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32")])
def test_wgrad_writes_only_its_columns(ws, kn, dtype, out):
    k, n = kn
    sizes = [130, 0, 77]
    off = offsets_of(sizes)
    a, dc = draw((sum(sizes), k), dtype, 108), draw((sum(sizes), n), dtype, 109)
    full = torch.full((3, k + 2, (n + 15) // 8 * 8), 9.0, dtype=DT[out], device="cuda")
    T.grouped_wgrad(a, dc, off, out=full[:, 1:k + 1, :n], workspace=ws)
    T.check(ws)
    ref, bound = OO.wgrad(f64(a), f64(dc), off.tolist())
    assert_close(full[:, 1:k + 1, :n], ref, bound, out, rel16(max(sizes)))
    full[:, 1:k + 1, :n] = 9.0
    assert bool((full == 9.0).all())


@pytest.mark.parametrize("k", [16, 128, 200, 384, 512, 640])
def test_many_large_tiles_of_few_k_blocks(ws, k):
    # Every pair of CTAs walks many units, each only a few K blocks long.
    m, n = 9000, 5000
    a8, sa, b8, sb = fp8_operands(m, n, k, 110)
    off = offsets_of([4000, 0, 5000])
    w8, sw = T.quantize_fp8(draw((3, n, k), "f32", 111), block_rows=128)
    a, w = draw((m, k), "bf16", 112), draw((3, k, n), "bf16", 113)
    dense = T.gemm_fp8(a8, sa, b8, sb, workspace=ws)
    T.check(ws)
    grouped8 = T.grouped_gemm_fp8(a8, sa, w8, sw, off, workspace=ws)
    T.check(ws)
    grouped = T.grouped_gemm(a, w, off, workspace=ws)
    T.check(ws)
    for rows, e in ((slice(0, 300), 0), (slice(3900, 4000), 0), (slice(8700, 9000), 2)):
        ref, bound = dev_fp8(a8[rows], sa[rows], b8, sb)
        assert_close_dev(dense[rows], ref, bound, "bf16", rel8(k))
        ref, bound = dev_fp8(a8[rows], sa[rows], w8[e], sw[e])
        assert_close_dev(grouped8[rows], ref, bound, "bf16", rel8(k))
        x, y = a[rows].double(), w[e].double()
        assert_close_dev(grouped[rows], x @ y, x.abs() @ y.abs(), "bf16", rel16(k))


def test_results_past_32_bit_offsets(ws):
    # More than 2^31 elements of the result; its last rows are compared.
    m, n, k = 530000, 4104, 64
    a8, sa, b8, sb = fp8_operands(m, n, k, 107)
    c = T.gemm_fp8(a8, sa, b8, sb, out_dtype="bf16", workspace=ws)
    T.check(ws)
    for rows in (slice(0, 130), slice(523000, 523600), slice(m - 300, m)):
        ref, bound = dev_fp8(a8[rows], sa[rows], b8, sb)
        assert_close_dev(c[rows], ref, bound, "bf16", rel8(k))
    q, s, _ = T.rmsnorm_fp8(c[:, :4096], torch.ones(4096, dtype=torch.bfloat16, device="cuda"))
    tail = c[m - 5:, :4096].double()
    want = tail / (tail.square().mean(1, keepdim=True) + 1e-6).sqrt()
    got = q[m - 5:].double() * s[m - 5:].double().repeat_interleave(128, 1)
    peak = want.abs().reshape(5, 32, 128).amax(2).repeat_interleave(128, 1)
    # e4m3 rounds by at most 2^-4 of a value and, below 2^-6, by 2^-10.
    assert bool(((got - want).abs() <= want.abs() * 0.0626 + peak / 448 * 2.0 ** -9).all())


@pytest.mark.parametrize("k", [1, 7, 130, 203, 1003])
@pytest.mark.parametrize("sizes", [[5, 0, 9], [700, 0, 2100]], ids=["few", "large"])
def test_what_lies_between_the_rows_is_not_read(ws, sizes, k):
    # Row lengths that end inside 16 bytes, with not-a-numbers up to the pitch.
    n, t = 1104 if sizes[0] > 100 else 136, sum(sizes)
    off = offsets_of(sizes)
    pad = (k + 23) // 8 * 8

    def apart(x, pitch):
        wide = torch.full((*x.shape[:-1], pitch), float("nan"), dtype=x.dtype, device="cuda")
        wide[..., : x.shape[-1]] = x
        return wide[..., : x.shape[-1]]

    a = apart(draw((t, k), "bf16", 114), pad)
    w = draw((3, n, k), "bf16", 115)
    kn = w.transpose(1, 2).contiguous()
    ref, bound = dev_grouped(a, w, off.tolist(), True)
    c = T.grouped_gemm(a, apart(w, pad), off, trans_b=True, out_dtype="f32", workspace=ws)
    T.check(ws)
    assert_close_dev(c, ref, bound, "f32", rel16(k))
    c = T.grouped_gemm(a, kn, off, out_dtype="f32", workspace=ws)
    T.check(ws)
    assert_close_dev(c, ref, bound, "f32", rel16(k))
    da = T.grouped_wgrad(a, apart(draw((t, n - 3), "bf16", 116), n + 8), off, out_dtype="f32",
                         workspace=ws)
    T.check(ws)
    assert bool(da.isfinite().all())

    pad8 = (k + 31) // 16 * 16
    a8, sa = T.quantize_fp8(draw((t, k), "f32", 117))
    b8, sb = T.quantize_fp8(draw((3, n, k), "f32", 118), block_rows=128)
    as_bytes = torch.full((t, pad8), 0x7f, dtype=torch.uint8, device="cuda")
    as_bytes[:, :k] = a8.view(torch.uint8)
    a8 = as_bytes.view(torch.float8_e4m3fn)[:, :k]
    as_bytes = torch.full((3, n, pad8), 0x7f, dtype=torch.uint8, device="cuda")
    as_bytes[:, :, :k] = b8.view(torch.uint8)
    b8 = as_bytes.view(torch.float8_e4m3fn)[:, :, :k]
    c = T.grouped_gemm_fp8(a8, sa, b8, sb, off, out_dtype="f32", workspace=ws)
    T.check(ws)
    for e, (lo, hi) in enumerate(zip(off.tolist()[:-1], off.tolist()[1:])):
        if hi > lo:
            ref, bound = dev_fp8(a8[lo:hi], sa[lo:hi], b8[e], sb[e])
            assert_close_dev(c[lo:hi], ref, bound, "f32", rel8(k))
