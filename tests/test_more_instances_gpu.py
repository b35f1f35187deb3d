"""GPU parity of the instances of the layer-norm, routing and clipping kernels that only
larger calls reach: dispatch of many rows that start anywhere, 8-bit layer norm of such
rows with a residual, long rows off 16 bytes, sorts of hundreds of thousands of pairs
up to the limit, and clips of 100 MB and more in few and in very many tensors.  The
definitions are computed on the GPU, in float64 where there is arithmetic.

Tolerances, from the kernels' arithmetic (fp32; a rounding to a type is off by at most
half a spacing, 2^-4, 2^-11, 2^-8 or 2^-24 of the value, 2^-25 in fp16's subnormals):
  - a layer norm's row of n columns: at most (n / 1024 rounded up to 8 more + 32)
    additions in a chain, under 80 for 40001 columns: 2^-17 of the sum of magnitudes; the
    corrected mean leaves d within 2^-23 |h| + 2^-22 |d| + 2^-17 mean|d|, and rstd within
    2^-16 of itself;
  - a norm over tensors: 34 * 2^-24 of itself whatever their number (a thread's sums
    keep what their additions round off, the rest are levels of lanes and warps); a
    scaled element four roundings more, and its own."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402

F32 = torch.float32
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": F32, "e4m3": torch.float8_e4m3fn}
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, F32: 2.0 ** -24}


def normals(n, seed, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, generator=g, device="cuda") + mean


def placed(rows, cols, dtype, seed, more=0, shift=0, mean=0.0):
    """A matrix whose rows lie `more` elements apart, from element `shift` on, and all the
    memory around it."""
    full = normals(rows * (cols + more) + shift + 40, seed, mean).to(DT[dtype])
    return full, full[shift:shift + rows * (cols + more)].view(rows, -1)[:, :cols]


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def untouched(full, view, before):
    """Whether all of `full` but the view is as it was."""
    mask = torch.zeros(full.shape, dtype=torch.bool, device="cuda")
    mask[view.storage_offset() - full.storage_offset():][:view.shape[0] * view.stride(0)] \
        .view(view.shape[0], -1)[:, :view.shape[1]] = True
    return torch.equal(bits(full)[~mask], bits(before)[~mask])


def within(got, ref, slack):
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    err = (got.double() - ref).abs()
    tol = ref.abs() * HALF[got.dtype] + tiny + slack * (1 + 2.0 ** -8)
    assert bool((err <= tol).all()), f"worst error/tolerance {float((err / tol).max())}"


# ---- dispatch of many rows that start anywhere --------------------------------------------

# Rows (in bytes) of 17 pieces and of more, with pieces enough for the instance of four
# pieces a thread; 16 pieces and a few rows less, which go to the other.  Choices 1, 3, 9.
MANY = [(20000, 1, 243), (7000, 3, 243), (7000, 3, 257), (21000, 1, 241), (2500, 1, 2002),
        (900, 3, 2002), (300, 9, 2006), (120, 9, 9004), (35, 9, 16010), (2400, 1, 2014)]


@pytest.mark.parametrize("x_at,out_at", [((0, 0), (0, 0)), ((1, 1), (3, 2)), ((2, 5), (1, 3)), ((5, 3), (0, 7))],
                         ids=str)
@pytest.mark.parametrize("dtype", ["f16", "f32", "e4m3"])
@pytest.mark.parametrize("tokens,k,row_bytes", MANY)
def test_dispatch_of_many_rows_that_start_anywhere(tokens, k, row_bytes, dtype, x_at, out_at):
    size = DT[dtype].itemsize
    cols = max(row_bytes // size, 1)
    rows = tokens * k + 3
    _, x = placed(tokens, cols, dtype, 1, *x_at)
    full, out = placed(rows, cols, dtype, 2, *out_at)
    before = full.clone()
    g = torch.Generator(device="cuda").manual_seed(3)
    slots = torch.randperm(tokens * k, generator=g, device="cuda").int().view(tokens, k)
    slots[torch.rand((tokens, k), generator=g, device="cuda") < 0.1] = -1
    slots[tokens // 2, 0] = rows + 7                     # past the rows: nobody's
    want = bits(out).clone()
    t, j = torch.nonzero((slots >= 0) & (slots < rows), as_tuple=True)
    want[slots[t, j].long()] = bits(x)[t]
    assert T.expert_dispatch(x, slots, out=out) is out
    assert torch.equal(bits(out), want) and untouched(full, out, before)


def test_dispatch_of_many_8_bit_rows_that_start_anywhere_with_their_scales():
    tokens, k, cols = 1500, 4, 1001
    q, s = T.quantize_fp8(normals(tokens * cols, 4).view(tokens, cols).bfloat16())
    q = q.contiguous()                                   # rows of 1001 bytes
    slots = torch.randperm(tokens * k, device="cuda").int().view(tokens, k)
    out, scales = T.expert_dispatch(q, slots, scales=s)
    at = slots.long().reshape(-1)
    assert torch.equal(bits(out)[at], bits(q).repeat_interleave(k, 0))
    assert torch.equal(scales[at], s.repeat_interleave(k, 0))


# ---- layer norm -----------------------------------------------------------------------------


def plain_norm(x, w, b, r):
    h = x.double() if r is None else x.double() + r.double()
    d = h - h.mean(1, keepdim=True)
    rstd = ((d * d).mean(1, keepdim=True) + 1e-5).rsqrt()
    y = d * rstd * w.double() + b.double()
    off = 2.0 ** -23 * h.abs() + 2.0 ** -22 * d.abs() + 2.0 ** -17 * d.abs().mean(1, keepdim=True)
    slack = off * rstd * w.double().abs() + 2.0 ** -16 * d.abs() * rstd * w.double().abs() + 2.0 ** -22 * y.abs()
    return y, h, slack


def check_fp8(q, s, y, slack):
    rows, cols = y.shape
    spread = s.double().repeat_interleave(128, 1)[:, :cols]
    err = (q.double() * spread - y).abs()
    assert bool((err <= y.abs() * 2.0 ** -4 + spread * 2.0 ** -10 + slack * 1.1 + y.abs() * 2.0 ** -21).all())

    def most(t):
        return torch.nn.functional.pad(t, (0, -cols % 128)).view(rows, -1, 128).amax(2)
    assert bool(((s.double() * 448 - most(y.abs())).abs() <= most(slack) + 2.0 ** -21 * most(y.abs())).all())


# Rows at a time of a block 2, 16, 1, 5 and 2, four times 152 blocks' worth and more.
@pytest.mark.parametrize("x_at,r_at,h_at", [((0, 0), (0, 0), None), ((1, 3), (2, 0), (5, 1)), ((8, 7), (3, 5), (1, 2))],
                         ids=str)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1300, 4001), (9800, 301), (620, 8191), (3100, 1501), (1250, 2760)])
def test_8_bit_norm_with_residual_of_rows_that_start_anywhere(rows, cols, dtype, x_at, r_at, h_at):
    if cols % 8 == 0 and x_at == (0, 0):
        x_at = (0, 1)                                    # these would start on 16 bytes
    x, r = placed(rows, cols, dtype, 5, *x_at, mean=0.5)[1], placed(rows, cols, dtype, 6, *r_at, mean=-0.25)[1]
    w, b = normals(cols, 7).to(DT[dtype]), normals(cols + 1, 8).to(DT[dtype])[1:]
    y, h64, slack = plain_norm(x, w, b, r)
    hfull, h_out = placed(rows, cols, dtype, 9, *h_at) if h_at else (None, None)
    before = None if hfull is None else hfull.clone()
    q, s, h = T.layernorm_fp8(x, w, b, residual=r, h_out=h_out)
    check_fp8(q, s, y, slack)
    within(h, h64, 2.0 ** -24 * h64.abs())
    if hfull is not None:
        assert h is h_out and untouched(hfull, h_out, before)
    # Bytes of y that start anywhere, scales row by row, the residual in place.
    odd = torch.zeros(rows * (cols + 2) + 1, dtype=torch.uint8, device="cuda").view(DT["e4m3"])
    odd = odd[1:].view(rows, cols + 2)[:, :cols]
    given = torch.empty((rows, s.shape[1]), device="cuda")
    q2, s2, h2 = T.layernorm_fp8(x, w, b, residual=r, out=odd, scales=given, h_out=r)
    assert q2 is odd and s2 is given and h2 is r
    assert torch.equal(bits(q2), bits(q)) and torch.equal(s2, s) and torch.equal(bits(r), bits(h))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(3, 8203), (200, 12288), (160, 16384), (3, 16386), (160, 32768), (3, 32771),
                                       (3, 40001)])
def test_norm_of_long_rows(rows, cols, dtype):
    x, r = placed(rows, cols, dtype, 10, mean=0.5)[1], placed(rows, cols, dtype, 11, mean=-1.0)[1]
    w, b = normals(cols, 12).to(DT[dtype]), normals(cols, 13).to(DT[dtype])
    for res in (None, r):
        y, h64, slack = plain_norm(x, w, b, res)
        got, h = T.layernorm(x, w, b, residual=res)
        within(got, y, slack)
        if res is not None:
            within(h, h64, 2.0 ** -24 * h64.abs())
        q, s, _ = T.layernorm_fp8(x, w, b, residual=res)
        check_fp8(q, s, y, slack)


# ---- sorts --------------------------------------------------------------------------------


def check_sort(ids, groups):
    """Against PyTorch's stable sort."""
    slots, offsets, order = T.expert_sort(ids, groups)
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < groups), flat, groups)
    want = torch.sort(key, stable=True)[1]
    n = int((key < groups).sum())
    assert torch.equal(order[:n].long(), want[:n]) and bool((order[n:] == -1).all())
    count = torch.bincount(key, minlength=groups + 1)[:groups]
    assert int(offsets[0]) == 0 and torch.equal(offsets[1:].long(), count.cumsum(0))
    place = torch.full_like(flat, -1)
    place[want[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(slots.reshape(-1).long(), place) and slots.shape == ids.shape


# Pairs a thread 2 and 4, 4 and 8, 8 and 16 on both sides of where they change, and the
# most pairs that a sort takes; groups with and without the launch that adds up counts.
@pytest.mark.parametrize("groups", [2, 60, 4096])
@pytest.mark.parametrize("tokens,k", [(311296, 1), (311297, 1), (100003, 4), (622592, 1), (622593, 1), (100001, 7),
                                      (1245184, 1), (1245185, 1), (250007, 6), (1 << 21, 8)])
def test_sort_of_many_pairs(tokens, k, groups):
    g = torch.Generator(device="cuda").manual_seed(14)
    ids = torch.randint(-1, groups + 1, (tokens, k), generator=g, device="cuda")
    check_sort(ids, groups)
    ids = ids.int()
    ids[torch.rand((tokens, k), generator=g, device="cuda") < 0.9] = groups - 1
    check_sort(ids, groups)
    check_sort(torch.full_like(ids, groups - 1), groups)
    with pytest.raises(T.TilesError):
        T.expert_sort(torch.zeros(((1 << 24) + 1, 1), dtype=torch.int32, device="cuda"), groups)


# ---- clips ---------------------------------------------------------------------------------

# Over 20 MB the kernels take 32 KB chunks; what is over 100 MB from the end is read past
# L2; 16, 120 and 1000 tensors go with a launch.
CLIPS = {
    "16 tensors": [5000003 + 4096 * i for i in range(16)],
    "48 tensors": [1500001 + 7777 * (i % 13) for i in range(48)],
    "120 tensors": [600001 + 16384 * (i % 3) for i in range(120)],
    "121 tensors": [600001 + 16383 * (i % 3) for i in range(121)],
    "1000 tensors": [70000 + i % 5 for i in range(1000)],
    "1100 tensors": [70001 + 16 * (i % 7) for i in range(1100)],
    "2500 tensors": [30001 + i % 17 for i in range(2500)],
    "one between small ones": [1] * 40 + [70000001] + [0, 3] * 40,
}


def gradients(sizes, shift):
    types = [torch.bfloat16, torch.float16, F32, torch.bfloat16]
    total = sum(sizes)
    base = normals(total + shift * len(sizes), 15) * 0.125
    out, at = [], 0
    for i, n in enumerate(sizes):
        out.append(base[at:at + n + shift].to(types[i % 4])[shift:])
        at += n + shift
    return out


def norm64(grads):
    return float(sum((g.double() ** 2).sum() for g in grads).sqrt())


@pytest.mark.parametrize("shift,shift_out", [(0, None), (0, 0), (3, None), (1, 2)])
@pytest.mark.parametrize("name", CLIPS)
def test_clip_of_much(name, shift, shift_out):
    grads = gradients(CLIPS[name], shift)
    before = [g.clone() for g in grads]
    want = norm64(grads)
    rel = 34 * 2.0 ** -24
    assert abs(float(T.grad_norm(grads)) - want) <= rel * want
    full = out = None
    if shift_out is not None:
        full = [torch.full((g.numel() + shift_out + 9,), 7.0, dtype=g.dtype, device="cuda") for g in grads]
        out = [f[shift_out:shift_out + g.numel()] for f, g in zip(full, grads)]
    norm = T.clip_grads(grads, 0.37 * want, out=out)
    assert abs(float(norm) - want) <= rel * want
    factor = 0.37 * want / (want + 1e-6)
    for i, g in enumerate(before):
        ref = g.double() * factor
        within(grads[i] if out is None else out[i], ref, (rel + 4 * 2.0 ** -24) * ref.abs())
        if out is not None:
            assert torch.equal(grads[i], g)
            assert bool((full[i][:shift_out] == 7.0).all()) and bool((full[i][shift_out + g.numel():] == 7.0).all())


@pytest.mark.parametrize("name", ["16 tensors", "48 tensors", "1100 tensors"])
@pytest.mark.parametrize("odd", [1e25, 1e13, 1e-30])
def test_clip_of_much_with_elements_whose_squares_leave_the_range(name, odd):
    # In the first tensor, which is read past L2, and in the last, which is not.
    grads = [g.float() * (1e-25 if odd < 1 else 1.0) for g in gradients(CLIPS[name], 0)]
    for g in (grads[0], grads[-1]):
        g[5::1009] = odd
    want = norm64(grads)
    before = [g.double() for g in (grads[0], grads[-1])]
    norm = T.clip_grads(grads, 0.5 * want)
    assert abs(float(norm) - want) <= 34 * 2.0 ** -24 * want
    factor = 0.5 * want / (want + 1e-6)
    for g, b in zip((grads[0], grads[-1]), before):
        within(g, b * factor, 38 * 2.0 ** -24 * (b * factor).abs() + 2.0 ** -149)


@pytest.mark.parametrize("where", [0, -1])
def test_clip_of_much_with_a_nan_or_an_infinity(where):
    for odd in (float("inf"), float("nan")):
        grads = gradients(CLIPS["1100 tensors"], 0)
        grads[where][-1] = odd
        assert str(float(T.clip_grads(grads, 1.0))) == str(odd)
        for i, g in enumerate(grads):
            if odd != odd:
                assert bool(g.isnan().all())
            else:
                assert not g[:-1].any() and (bool(g[-1].isnan()) if i == where % len(grads) else not g[-1].any())


def test_clips_of_much_give_the_same_bits_and_leave_small_norms_alone():
    grads = gradients(CLIPS["121 tensors"], 0)
    first = T.grad_norm(grads)
    out = [torch.empty_like(g) for g in grads]
    for _ in range(3):
        assert torch.equal(T.clip_grads(grads, 1.0, out=out), first)
    before = [g.clone() for g in grads]
    assert torch.equal(T.clip_grads(grads, 2 * float(first)), first)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
