"""GPU parity of the expert sort, dispatch, weighted sum and its gradients with
the float64 definitions.

The sort and the dispatch are exact.  The sum adds k products in fp32 (each
fused into the addition: k + 1 roundings of at most 2^-24 of the magnitudes)
and rounds once, by at most half a spacing.  A row's gradient is one fp32
product, rounded once more.  A weight's gradient adds at most cols / 64 terms
a thread and 12 levels of threads."""

import numpy as np
import pytest

from oracle import operators as OO
from oracle import tolerance as OT

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
      "e4m3": torch.float8_e4m3fn}


def ids_of(tokens, k, groups, seed, low=0, favourite=None, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(low, groups - low, (tokens, k), generator=g)
    if favourite is not None:
        ids[torch.rand((tokens, k), generator=g) < 0.9] = favourite
    return ids.to(dtype).cuda()


def plain_sort(ids, groups):
    """The definition by a stable sort on the host (quick where there are many pairs)."""
    flat = ids.cpu().reshape(-1).to(torch.int64).numpy()
    key = np.where((flat >= 0) & (flat < groups), flat, groups)
    order = np.argsort(key, kind="stable")
    n = int((key < groups).sum())
    slots = np.empty(flat.size, np.int64)
    slots[order] = np.arange(flat.size)
    slots[key == groups] = -1
    order[n:] = -1
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=groups + 1)[:groups])])
    return slots.reshape(ids.shape), offsets, order


def assert_sorted(got, ids, groups):
    for name, t, want in zip(("slots", "offsets", "order"), got, plain_sort(ids, groups)):
        assert t.dtype == torch.int32 and t.shape == want.shape, name
        assert np.array_equal(t.cpu().numpy(), want), name


SORTS = [(1, 1, 1), (1, 8, 16), (16, 4, 16), (7, 3, 5), (33, 2, 3), (100, 8, 256), (1, 1, 4096),
         (511, 8, 4095), (512, 8, 64), (513, 8, 64), (4096, 1, 7), (4097, 1, 7), (1025, 1, 60),
         (5000, 6, 60), (16384, 8, 64), (16384, 8, 1024), (16384, 8, 1025), (9999, 7, 4096),
         (30011, 8, 33), (70000, 4, 2), (200003, 6, 128)]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=str)
@pytest.mark.parametrize("tokens,k,groups", SORTS)
def test_sort(tokens, k, groups, dtype):
    ids = ids_of(tokens, k, groups, tokens + k, dtype=dtype)
    assert_sorted(T.expert_sort(ids, groups), ids, groups)


@pytest.mark.parametrize("tokens,k,groups", [(9, 2, 4), (600, 8, 40), (3000, 8, 40), (16384, 8, 300)])
def test_sort_leaves_out_ids_that_are_no_experts(tokens, k, groups):
    ids = ids_of(tokens, k, groups, 1, low=-3)            # from -3 to groups + 2
    assert int((ids < 0).sum()) and int((ids >= groups).sum())
    assert_sorted(T.expert_sort(ids, groups), ids, groups)
    # Ids that only 64 bits hold: their low words are experts.
    far = ids + (ids % 2) * (1 << 32) - (ids % 3) * (1 << 40)
    assert_sorted(T.expert_sort(far, groups), far, groups)
    none = torch.full_like(ids, -1)
    assert_sorted(T.expert_sort(none, groups), none, groups)
    one = torch.full_like(ids, groups - 1)
    assert_sorted(T.expert_sort(one, groups), one, groups)


@pytest.mark.parametrize("tokens", [50, 16384])
def test_sort_of_a_favourite_expert_and_of_repeated_ones(tokens):
    ids = ids_of(tokens, 8, 64, 2, favourite=63)
    assert_sorted(T.expert_sort(ids, 64), ids, 64)


@pytest.mark.parametrize("tokens", [20, 5000])
def test_sort_of_strided_ids_and_with_a_given_workspace(tokens):
    full = ids_of(tokens, 11, 16, 3)
    ids = full[:, 2:8]
    need = T.load().tiles_expert_sort_workspace_bytes(tokens, 6, 16)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert_sorted(T.expert_sort(ids, 16, workspace=ws), ids, 16)
    assert bool((ws[:256] == 255).all()) and bool((ws[need:] == 255).all())
    if need > 256:
        with pytest.raises(T.TilesError, match="workspace"):
            T.expert_sort(ids, 16, workspace=ws[:need - 1])


def test_sort_of_no_tokens():
    slots, offsets, order = T.expert_sort(torch.empty((0, 4), dtype=torch.int64, device="cuda"), 5)
    assert slots.shape == (0, 4) and offsets.tolist() == [0] * 6 and order.shape == (0,)


# ---- rows -----------------------------------------------------------------------------------


def draw(shape, dtype, seed, pitch=None, shift=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols = shape
    pitch = pitch or cols
    full = torch.randn(rows * pitch + shift, generator=g, device="cuda") * scale
    return full.to(DT[dtype])[shift:].view(rows, pitch)[:, :cols]


def f64(t):
    return t.double().cpu().numpy()


def within(got, ref, slack, dtype):
    err = np.abs(f64(got) - ref)
    tol = OT.ulp(ref, dtype) / 2 * (1 + 2.0 ** -6) + slack
    assert np.all(err <= tol), f"worst error/tolerance {np.max(err / tol)}"


def routed(tokens, k, groups, seed, low=-1):
    """Slots of a sort with some pairs left out."""
    ids = ids_of(tokens, k, groups, seed, low=low)
    return T.expert_sort(ids, groups)[0]


ROWS = [(1, 1, 8), (1, 8, 4096), (3, 2, 1), (5, 3, 7), (40, 4, 64), (33, 6, 100), (7, 2, 129),
        (9, 8, 3000), (6, 11, 200), (4, 20, 4104), (300, 8, 256), (5, 3, 9000), (2, 2, 40001),
        (700, 2, 33)]


@pytest.mark.parametrize("dtype", ["f16", "f32", "e4m3"])
@pytest.mark.parametrize("tokens,k,cols", ROWS)
def test_dispatch(tokens, k, cols, dtype):
    x, slots = draw((tokens, cols), dtype, 1), routed(tokens, k, 5, 2)
    got = T.expert_dispatch(x, slots)
    assert got.shape == (tokens * k, cols) and got.dtype == x.dtype
    want = OO.expert_dispatch(f64(x), slots.cpu().numpy(), tokens * k)
    named = ~np.isnan(want[:, 0])
    assert np.array_equal(f64(got)[named], want[named])
    # Into a given matrix: rows that no slot names stay as they are.
    full = torch.full((tokens * k + 2, cols + 3), 2.0, device="cuda").to(x.dtype)
    out = T.expert_dispatch(x, slots, out=full[:, :cols])
    want = OO.expert_dispatch(f64(x), slots.cpu().numpy(), tokens * k + 2, fill=2.0)
    assert np.array_equal(f64(out), want)
    assert bool((full[:, cols:].float() == 2.0).all())


@pytest.mark.parametrize("by_block_in", [True, False])
@pytest.mark.parametrize("by_block_out", [True, False, None])
@pytest.mark.parametrize("tokens,k,cols", [(1, 4, 4096), (37, 3, 200), (500, 8, 1000), (3, 2, 100)])
def test_dispatch_of_8_bit_rows_with_their_scales(tokens, k, cols, by_block_in, by_block_out):
    q, s = T.quantize_fp8(draw((tokens, cols), "bf16", 3))
    if not by_block_in:
        s = s.contiguous()
    slots, n = routed(tokens, k, 7, 4), tokens * k
    nb = s.shape[1]
    given = None if by_block_out is None else \
        torch.full((nb, n), 5.0, device="cuda").t() if by_block_out else \
        torch.full((n, nb), 5.0, device="cuda")
    rows, scales = T.expert_dispatch(q, slots, scales=s, scales_out=given)
    assert scales.shape == (n, nb) and (given is None or scales is given)
    sl = slots.cpu().numpy()
    for got, want in ((rows, OO.expert_dispatch(f64(q), sl, n)),
                      (scales, OO.expert_dispatch(f64(s), sl, n))):
        named = ~np.isnan(want[:, 0])
        assert np.array_equal(f64(got)[named], want[named])
        if got is given:
            assert bool((got[torch.tensor(~named, device="cuda")] == 5.0).all())


@pytest.mark.parametrize("shift,pitch", [(0, 128), (1, 131), (8, 160), (4, 132), (2, 130)])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
def test_dispatch_of_strided_and_unaligned_rows(shift, pitch, dtype):
    x, slots = draw((50, 128), dtype, 5, pitch=pitch, shift=shift), routed(50, 3, 6, 6)
    full = torch.full((150, 140), 2.0, device="cuda").to(x.dtype)
    out = T.expert_dispatch(x, slots, out=full[:, 3:131])
    want = OO.expert_dispatch(f64(x), slots.cpu().numpy(), 150, fill=2.0)
    assert np.array_equal(f64(out), want)
    assert bool((full[:, :3].float() == 2.0).all()) and bool((full[:, 131:].float() == 2.0).all())


def test_dispatch_keeps_bits_and_passes_over_slots_out_of_range():
    x = torch.randint(0, 2 ** 31 - 1, (30, 64), device="cuda", dtype=torch.int32).view(torch.float32)
    slots = routed(30, 2, 4, 7, low=0)
    assert torch.equal(T.expert_dispatch(x, slots).view(torch.int32)[slots[:, 1].long()],
                       x.view(torch.int32))
    out = torch.full((20, 64), 3.0, device="cuda")        # 60 slots, 20 rows
    T.expert_dispatch(x, slots, out=out)
    named = slots.cpu().numpy()
    for t, j in np.ndindex(named.shape):
        if named[t, j] < 20:
            assert torch.equal(out[named[t, j]].view(torch.int32), x[t].view(torch.int32))
    wild = torch.tensor([[-5, 2 ** 31 - 1], [-2 ** 31, 20]], dtype=torch.int32, device="cuda")
    before = out.clone()
    T.expert_dispatch(x[:2], wild, out=out)
    assert torch.equal(out.view(torch.int32), before.view(torch.int32))
    assert not T.expert_combine(out, wild).any()


@pytest.mark.parametrize("dtype,weights", [("f16", "f32"), ("bf16", "bf16"), ("f32", "f16"),
                                           ("bf16", None)])
@pytest.mark.parametrize("tokens,k,cols", ROWS)
def test_combine(tokens, k, cols, dtype, weights):
    rows, slots = draw((tokens * k, cols), dtype, 8), routed(tokens, k, 5, 9)
    w = draw((tokens, k), weights, 10) if weights else None
    got = T.expert_combine(rows, slots, w)
    sl = slots.cpu().numpy()
    y, s = OO.expert_combine(f64(rows), sl, None if w is None else f64(w))
    within(got, y, (k + 1) * 2.0 ** -24 * s, dtype)
    assert bool((got[torch.tensor((sl < 0).all(1), device="cuda")] == 0).all())
    full = torch.full((tokens, cols + 5), 7.0, device="cuda").to(rows.dtype)
    out = T.expert_combine(rows, slots, w, out=full[:, :cols])
    assert torch.equal(out, got) and bool((full[:, cols:].float() == 7.0).all())


@pytest.mark.parametrize("dtype,weights", [("f16", "f32"), ("bf16", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("tokens,k,cols", ROWS)
def test_combine_gradients(tokens, k, cols, dtype, weights):
    n = tokens * k
    rows, slots = draw((n, cols), dtype, 11), routed(tokens, k, 5, 12)
    w, dy = draw((tokens, k), weights, 13), draw((tokens, cols), dtype, 14)
    drows, dw = T.expert_combine_grad(dy, rows, slots, w)
    assert drows.shape == rows.shape and drows.dtype == rows.dtype and dw.dtype == torch.float32
    rr, rw, s = OO.expert_combine_grad(f64(dy), f64(rows), slots.cpu().numpy(), f64(w))
    named = ~np.isnan(rr[:, 0])
    within(drows[torch.tensor(named, device="cuda")], rr[named], 2.0 ** -24 * np.abs(rr[named]), dtype)
    within(dw, rw, (cols / 64 + 12) * 2.0 ** -24 * s, "f32")
    full, wide = torch.full((n, cols + 5), 7.0, device="cuda").to(rows.dtype), \
        torch.full((tokens, k + 3), 7.0, device="cuda")
    full[:, :cols] = 3.0
    a, b = T.expert_combine_grad(dy, rows, slots, w, drows_out=full[:, :cols], dweights_out=wide[:, :k])
    assert torch.equal(a[torch.tensor(named, device="cuda")], drows[torch.tensor(named, device="cuda")])
    # (Rows that start elsewhere may be added in another order: the same bound, not the same bits.)
    within(b, rw, (cols / 64 + 12) * 2.0 ** -24 * s, "f32")
    assert bool((a[torch.tensor(~named, device="cuda")].float() == 3.0).all())
    assert bool((full[:, cols:].float() == 7.0).all()) and bool((wide[:, k:] == 7.0).all())


@pytest.mark.parametrize("shift,pitch", [(1, 131), (8, 160), (4, 130)])
def test_combine_of_strided_rows_slots_and_weights(shift, pitch):
    rows = draw((90, 128), "bf16", 15, pitch=pitch, shift=shift)
    ids = ids_of(30, 3, 4, 16)
    wide = torch.full((30, 5), -7, dtype=torch.int32, device="cuda")
    wide[:, 1:4] = T.expert_sort(ids, 4)[0]
    slots, w = wide[:, 1:4], draw((30, 3), "f32", 17, pitch=8)
    dy = draw((30, 128), "bf16", 18, pitch=pitch)
    sl = slots.cpu().numpy()
    y, s = OO.expert_combine(f64(rows), sl, f64(w))
    within(T.expert_combine(rows, slots, w), y, 4 * 2.0 ** -24 * s, "bf16")
    drows, dw = T.expert_combine_grad(dy, rows, slots, w)
    rr, rw, s = OO.expert_combine_grad(f64(dy), f64(rows), sl, f64(w))
    within(drows, rr, 2.0 ** -24 * np.abs(rr), "bf16")
    within(dw, rw, 14 * 2.0 ** -24 * s, "f32")


def test_what_a_left_out_choice_holds_does_not_matter():
    rows, w = draw((8, 64), "bf16", 19), torch.ones((2, 2), device="cuda")
    slots = torch.tensor([[0, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    w[0, 1] = w[1, 0] = float("nan")
    w[1, 1] = float("inf")
    rows[1:] = float("nan")
    y = T.expert_combine(rows, slots, w)
    assert torch.equal(y[0], rows[0]) and not y[1].any()
    drows, dw = T.expert_combine_grad(rows[:1].expand(2, 64).contiguous(), rows, slots, w)
    assert torch.equal(drows[0], rows[0])
    assert dw[0, 1] == 0 and not dw[1].any() and float(dw[0, 0]) > 0
    # One that counts does.
    slots[1, 1] = 3
    assert bool(T.expert_combine(rows, slots, w)[1].isnan().all())


def test_the_same_row_may_be_added_twice():
    rows = draw((4, 96), "f32", 20)
    slots = torch.tensor([[2, 2]], dtype=torch.int32, device="cuda")
    assert torch.equal(T.expert_combine(rows, slots), rows[2:3] * 2)


def test_no_tokens_and_no_rows():
    none = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    x = torch.empty((0, 64), device="cuda")
    assert T.expert_dispatch(x, none).shape == (0, 64)
    assert T.expert_combine(torch.ones((5, 64), device="cuda"), none).shape == (0, 64)
    drows, dw = T.expert_combine_grad(x, x, none, torch.empty((0, 3), device="cuda"))
    assert drows.shape == (0, 64) and dw.shape == (0, 3)
    # Tokens without a row in reach.
    slots = torch.full((4, 3), -1, dtype=torch.int32, device="cuda")
    assert not T.expert_combine(x, slots).any()
    dy, w = torch.ones((4, 64), device="cuda"), torch.ones((4, 3), device="cuda")
    _, dw = T.expert_combine_grad(dy, x, slots, w)
    assert dw.shape == (4, 3) and not dw.any()


def test_rows_past_32_bits_of_elements():
    # 600,000 x 4096 e4m3 rows: 2.4e9 elements; the last rows are where they belong.
    tokens, cols, k = 300000, 4096, 2
    x = torch.zeros((tokens, cols), dtype=torch.uint8, device="cuda")
    x[-3:] = torch.randint(0, 120, (3, cols), device="cuda", dtype=torch.uint8)
    slots = torch.arange(tokens * k, dtype=torch.int32, device="cuda").view(tokens, k)
    out = T.expert_dispatch(x.view(torch.float8_e4m3fn), slots).view(torch.uint8)
    assert torch.equal(out[-6:], x[-3:].repeat_interleave(2, 0)) and not out[:-6].any()
    del x
    rows = out.view(torch.float16)                        # 600,000 x 2048
    y = T.expert_combine(rows, slots)
    assert torch.equal(y[-3:], (rows[-6::2].float() * 2).half()) and not y[:-3].any()


def test_repeated_calls_give_the_same_bits():
    ids = ids_of(3000, 6, 60, 21)
    slots, offsets, order = T.expert_sort(ids, 60)
    rows, w = draw((18000, 500), "bf16", 22), torch.rand((3000, 6), device="cuda")
    dy = draw((3000, 500), "bf16", 23)
    first = (slots, offsets, order, T.expert_combine(rows, slots, w),
             *T.expert_combine_grad(dy, rows, slots, w))
    for _ in range(3):
        again = (*T.expert_sort(ids, 60), T.expert_combine(rows, slots, w),
                 *T.expert_combine_grad(dy, rows, slots, w))
        assert all(torch.equal(a, b) for a, b in zip(first, again))
