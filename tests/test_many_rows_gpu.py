"""GPU parity of the layer norm, the routing calls and the clipping where there
are many rows or many bytes: the kernels that keep the next rows on their way in
(from some hundred rows on), and the clip on both sides of what a chunk and a launch hold.
The plain forms are computed in float64 on the GPU.

Tolerances, from the kernels' arithmetic (fp32, one rounding to the output's
type of at most half a spacing, 2^-11, 2^-8 or 2^-24 of the value, 2^-25 in
fp16's subnormals):
  - a layer norm's row: a sum over n <= 8192 columns in a thread's 16, five or
    more levels of lanes and of warps, under 32 roundings of 2^-24 of the sum of
    magnitudes (2^-19); the corrected mean leaves d within 2^-23 |h| + 2^-22 |d|
    + 2^-18 mean|d|, and rstd within 2^-17 of itself;
  - the gradient has twice as many terms of the same kind: 2^-17 of the sums of
    magnitudes that enter it (a weight's gradient adds at most rows / 152 terms a
    thread, 64 partials a thread and a tree: 2^-16);
  - a weighted sum of k products: k + 1 roundings of 2^-24 of the magnitudes;
  - a dot product of n <= 8192 columns: 16 terms a thread and 9 levels, 2^-19;
  - a norm over many tensors: 2^-24 times 34 of itself, a scaled element two more
    roundings.
"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def draw(rows, cols, dtype, seed, mean=0.0, pitch=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pitch = pitch or cols
    full = (torch.randn(rows * pitch, generator=g, device="cuda") + mean).to(DT[dtype])
    return full.view(rows, pitch)[:, :cols]


def within(got, ref, slack=0.0):
    """One rounding of ref to got's type, and what was off before it."""
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    tol = ref.abs() * HALF[got.dtype] + tiny + slack * (1 + 2.0 ** -8)
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst error/tolerance {float((err / tol).max())}"


# ---- layer norm ---------------------------------------------------------------------------

# Rows at a time of a block 5, 2, 16, 4, 1, 1, 1 and 2, twice 152 blocks' worth and more,
# with and without a last round that not every block takes part in.
NORM = [(1600, 1304), (608, 4096), (5000, 264), (1217, 2048), (304, 8192), (471, 6000), (330, 5000), (700, 3200)]


def plain_norm(x, w, b, r, eps):
    h = x.double() if r is None else x.double() + r.double()
    d = h - h.mean(1, keepdim=True)
    u = (d * d).mean(1, keepdim=True) + eps
    rstd = u.rsqrt()
    y = d * rstd * w.double() + (0.0 if b is None else b.double())
    off = 2.0 ** -23 * h.abs() + 2.0 ** -22 * d.abs() + 2.0 ** -18 * d.abs().mean(1, keepdim=True)
    n = d.abs() * rstd * w.double().abs()
    slack = off * rstd * w.double().abs() + 2.0 ** -17 * n + 2.0 ** -22 * y.abs()
    return y, h, slack


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols", NORM)
@pytest.mark.parametrize("residual,bias", [(True, True), (False, True), (True, False)])
def test_norm(rows, cols, dtype, residual, bias):
    x = draw(rows, cols, dtype, 1, 0.5, cols + 8)
    r = draw(rows, cols, dtype, 2, -0.25, cols + 16) if residual else None
    w = draw(1, cols, "f32" if bias else dtype, 3)[0]
    b = draw(1, cols, "f32", 4)[0] if bias else None
    y64, h64, slack = plain_norm(x, w, b, r, 1e-5)
    out = torch.full((rows, cols + 24), 7.0, dtype=DT[dtype], device="cuda")
    y, h = T.layernorm(x, w, b, residual=r, out=out[:, :cols])
    within(y, y64, slack)
    assert bool((out[:, cols:] == 7.0).all())
    if residual:
        within(h, h64, 2.0 ** -24 * h64.abs())
    # 8 bits: half a step of the block's scale where the value is small, 2^-4 else.
    q, s, _ = T.layernorm_fp8(x, w, b, residual=r)
    spread = s.double().repeat_interleave(128, 1)[:, :cols]
    err = (q.double() * spread - y64).abs()
    assert bool((err <= y64.abs() * 2.0 ** -4 + spread * 2.0 ** -10 + slack * 1.1 +
                 y64.abs() * 2.0 ** -21).all())
    short = torch.nn.functional.pad(y64.abs(), (0, -cols % 128)).view(rows, -1, 128).amax(2)
    most = torch.nn.functional.pad(slack, (0, -cols % 128)).view(rows, -1, 128).amax(2)
    assert bool(((s.double() * 448 - short).abs() <= most + 2.0 ** -21 * short).all())
    # In place, and a copy of x without a residual.
    if residual:
        h2 = r.clone()
        y2, h3 = T.layernorm(x, w, b, residual=h2, h_out=h2)
        assert h3 is h2 and torch.equal(h2, h) and torch.equal(y2, y)
    else:
        copy = torch.empty_like(x)
        y2, h3 = T.layernorm(x, w, b, h_out=copy)
        assert h3 is copy and torch.equal(copy, x) and torch.equal(y2, y)


# Rows that start anywhere, four times 152 blocks' worth and more: rows at a time of a
# block 2, 16, 1, 5 and 2.  Pitches and offsets by which x, the residual and y start
# differently from one another, and even ones.
ODD = [(1300, 4001), (9800, 301), (620, 8191), (3100, 1501), (1250, 2760)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols", ODD)
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("more,shift", [((0, 0, 0), (0, 0, 0)), ((0, 0, 0), (1, 1, 1)), ((1, 2, 5), (3, 0, 6)),
                                        ((8, 3, 1), (7, 5, 2))], ids=str)
def test_norm_of_rows_that_start_anywhere(rows, cols, dtype, residual, more, shift):
    def view(i, seed, mean):
        full = draw(1, rows * (cols + more[i]) + shift[i] + 9, dtype, seed, mean)[0]
        return full, full[shift[i]:shift[i] + rows * (cols + more[i])].view(rows, -1)[:, :cols]
    x, r = view(0, 1, 0.5)[1], view(1, 2, -0.25)[1] if residual else None
    full, out = view(2, 3, 0.0)
    full.fill_(7.0)
    w, b = draw(1, cols, dtype, 4)[0], draw(1, cols + 1, dtype, 5)[0][1:]
    y64, h64, slack = plain_norm(x, w, b, r, 1e-5)
    y, h = T.layernorm(x, w, b, residual=r, out=out)
    within(y, y64, slack)
    keep = torch.ones_like(full, dtype=torch.bool)
    keep[shift[2]:shift[2] + rows * (cols + more[2])].view(rows, -1)[:, :cols] = False
    assert bool((full[keep] == 7.0).all())
    if residual:
        within(h, h64, 2.0 ** -24 * h64.abs())
        y2, h2 = T.layernorm(x, w, b, residual=r, h_out=r)
        assert h2 is r and torch.equal(r, h) and torch.equal(y2, y)
    q, s, _ = T.layernorm_fp8(x, w, b, residual=None)
    y64, _, slack = plain_norm(x, w, b, None, 1e-5)
    spread = s.double().repeat_interleave(128, 1)[:, :cols]
    err = (q.double() * spread - y64).abs()
    assert bool((err <= y64.abs() * 2.0 ** -4 + spread * 2.0 ** -10 + slack * 1.1 + y64.abs() * 2.0 ** -21).all())
    odd = torch.zeros(rows * (cols + 1) + 1, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    odd = odd[1:].view(rows, cols + 1)[:, :cols]
    q2, s2, _ = T.layernorm_fp8(x, w, b, out=odd)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


@pytest.mark.parametrize("rows,cols", [(1000, 4096), (1300, 4097)])
def test_norm_of_rows_with_nans_infinities_and_constants_between_others(rows, cols):
    x = draw(rows, cols, "bf16", 5)
    w, b = draw(1, cols, "bf16", 6)[0], draw(1, cols, "bf16", 7)[0]
    clean = T.layernorm(x, w, b)[0].clone()
    x[::7, 5] = float("nan")
    x[3::7, 4095] = float("inf")
    x[5::7] = 3.0
    y = T.layernorm(x, w, b)[0]
    assert bool(y[::7].isnan().all()) and bool(y[3::7].isnan().all())
    assert torch.equal(y[5::7], b.expand(len(y[5::7]), cols))
    rest = [i for i in range(rows) if i % 7 not in (0, 3, 5)]
    assert torch.equal(y[rest], clean[rest])
    s = T.layernorm_fp8(x, w, b)[1]
    assert bool(s[::7].isnan().all()) and not bool(s[rest].isnan().any())


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1600, 1304), (608, 4096), (5000, 264), (304, 8192), (700, 3200),
                                       (1700, 1301), (330, 5001), (200, 8191), (170, 12291), (170, 12296)])
def test_norm_gradients(rows, cols, dtype):
    h, dy = draw(rows, cols, dtype, 8, 0.5, cols + 8), draw(rows, cols, dtype, 9)
    dh, w = draw(rows, cols, dtype, 10), draw(1, cols, dtype, 11)[0]
    d = h.double() - h.double().mean(1, keepdim=True)
    r = ((d * d).mean(1, keepdim=True) + 1e-5).rsqrt()
    g = dy.double() * w.double()
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    want = (g - mean(g)) * r - d * mean(g * d) * r ** 3 + dh.double()
    size = (g.abs() + mean(g.abs())) * r + d.abs() * mean((g * d).abs()) * r ** 3 + \
        d.abs() * mean(g.abs()) * r * r + dh.double().abs()
    dx, dw, db = T.layernorm_grad(dy, h, w, dh=dh)
    within(dx, want, 2.0 ** -17 * size)
    e = dy.double() * d * r
    within(dw, e.sum(0), 2.0 ** -16 * (e.abs() + dy.double().abs()).sum(0))
    within(db, dy.double().sum(0), 2.0 ** -17 * dy.double().abs().sum(0))


# ---- routing ------------------------------------------------------------------------------


def routed(tokens, k, groups, seed):
    """Slots of a sort with every tenth pair or so left out; the rows that are somebody's."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, groups, (tokens, k), generator=g, device="cuda")
    ids[torch.rand((tokens, k), generator=g, device="cuda") < 0.1] = -1
    ids[tokens // 2] = -1                                # a token without any
    slots, offsets, _ = T.expert_sort(ids, groups)
    return slots, int(offsets[-1])


@pytest.mark.parametrize("dtype,weights", [("f16", "f32"), ("bf16", "bf16"), ("f32", "f16"), ("bf16", None)])
@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 6, 7, 8, 9])
@pytest.mark.parametrize("tokens,cols", [(5000, 520), (1300, 2056)])
def test_combine(tokens, cols, k, dtype, weights):
    if dtype == "f32":
        tokens = tokens // 2 + 1                         # a piece holds half as many columns
    slots, _ = routed(tokens, k, 16, k)
    rows = draw(tokens * k, cols, dtype, 1)
    nobody = torch.ones(tokens * k, dtype=torch.bool, device="cuda")
    nobody[slots[slots >= 0].long()] = False
    rows[nobody] = float("nan")                          # never read
    w = None if weights is None else draw(tokens, k, weights, 2)
    if w is not None:
        w[slots < 0] = float("nan")                      # neither
    y = T.expert_combine(rows, slots, w)
    ref = torch.zeros(tokens, cols, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for j in range(k):
        live = slots[:, j] >= 0
        p = rows[slots[live, j].long()].double()
        if w is not None:
            p = p * w[live, j:j + 1].double()
        ref[live] += p
        mag[live] += p.abs()
    within(y, ref, (k + 1) * 2.0 ** -24 * mag)
    assert bool((y[tokens // 2] == 0).all())


# Threads a token 32 (16 tokens a block), 160, 256, 288 and 512, and rows that go two
# pieces a thread or (more than four choices) to the kernel without the ring.
@pytest.mark.parametrize("dtype,weights", [("f16", "f32"), ("bf16", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 6, 7, 8, 9])
@pytest.mark.parametrize("tokens,pieces", [(5001, 17), (1000, 131), (700, 256), (650, 260), (304, 512), (311, 700)])
def test_combine_gradients(tokens, pieces, k, dtype, weights):
    cols = pieces * (4 if dtype == "f32" else 8)
    slots, used = routed(tokens, k, 16, k)
    rows, dy = draw(tokens * k, cols, dtype, 1), draw(tokens, cols, dtype, 2, 0.0, cols + 8)
    w = draw(tokens, k, weights, 3)
    w[slots < 0] = float("nan")
    out = torch.full_like(rows, 5.0)
    drows, dw = T.expert_combine_grad(dy, rows, slots, w, drows_out=out)
    assert drows is out and bool((out[used:] == 5.0).all())
    for j in range(k):
        live = slots[:, j] >= 0
        at = slots[live, j].long()
        want = dy[live].double() * w[live, j:j + 1].double()
        within(drows[at], want, 2.0 ** -24 * want.abs())
        e = dy[live].double() * rows[at].double()
        within(dw[live, j], e.sum(1), 2.0 ** -19 * e.abs().sum(1))
        assert bool((dw[~live, j] == 0).all())


@pytest.mark.parametrize("k", [1, 2, 4, 8, 9])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_dispatch(k, dtype):
    tokens, cols = 4001, 1040
    slots, used = routed(tokens, k, 33, k)
    x = draw(tokens, cols, "bf16", 1)
    scales = None
    if dtype == "e4m3":
        x, scales = T.quantize_fp8(x)
    out = torch.full((tokens * k, cols), 2.0, device="cuda").to(x.dtype)
    got = T.expert_dispatch(x, slots, scales=scales, out=out)
    t, j = torch.nonzero(slots >= 0, as_tuple=True)
    at = slots[t, j].long()
    raw = lambda m: m.view(torch.uint8 if dtype == "e4m3" else torch.int16)  # noqa: E731
    assert torch.equal(raw(out)[at], raw(x.contiguous())[t])
    assert bool((out[used:].float() == 2.0).all())
    if scales is not None:
        assert torch.equal(got[1][at], scales[t])


# ---- clipping -------------------------------------------------------------------------------

# Chunks are 8 KB, tensors 16, 120 and 1000 a launch: on both sides of those.
CLIPS = [[4096], [4097], [524288], [524280, 8], [8192] * 16, [8193] * 17, [8193] * 33, [1] * 64,
         [1] * 65, [1] * 121, [0, 3, 0], [262144, 262144], [262144, 262145],
         [700] * 1000, [700] * 1001, [3001] * 2003]


@pytest.mark.parametrize("sizes", CLIPS, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("shift,shift_out", [(0, None), (0, 0), (0, 1), (3, None), (3, 3), (3, 2)])
def test_clip(sizes, shift, shift_out):
    types = [torch.bfloat16, torch.float16, torch.bfloat16]
    grads = [draw(1, n + shift, "f32", i)[0].to(types[i % 3])[shift:] for i, n in enumerate(sizes)]
    before = [g.clone() for g in grads]
    norm64 = sum((g.double() ** 2).sum() for g in grads).sqrt()
    rel = 34 * 2.0 ** -24
    assert abs(float(T.grad_norm(grads)) - float(norm64)) <= rel * float(norm64)
    bound = 0.37 * float(norm64)
    full = None
    if shift_out is not None:
        full = [torch.full((g.numel() + shift_out + 9,), 7.0, dtype=g.dtype, device="cuda") for g in grads]
    out = full and [f[shift_out:shift_out + g.numel()] for f, g in zip(full, grads)]
    norm = T.clip_grads(grads, bound, out=out)
    assert abs(float(norm) - float(norm64)) <= rel * float(norm64)
    factor = bound / (float(norm64) + 1e-6)
    for i, g in enumerate(before):
        want = g.double() * factor
        got = grads[i] if out is None else out[i]
        within(got, want, (rel + 4 * 2.0 ** -24) * want.abs())
        if out is not None:
            assert torch.equal(grads[i], g)
            rest = torch.cat([full[i][:shift_out], full[i][shift_out + g.numel():]])
            assert bool((rest == 7.0).all())


@pytest.mark.parametrize("count", [1, 150])
def test_clip_of_much_with_elements_whose_squares_leave_the_range(count):
    n = 3000000 // count
    for scale, odd in ((1.0, 1e25), (1e-25, 1e-3), (1e-25, 1e-25), (1.0, 1e-30), (1e13, 1.0)):
        grads = [draw(1, n, "f32", i)[0] * scale for i in range(count)]
        grads[count // 2][5::1009] = odd
        norm64 = sum((g.double() ** 2).sum() for g in grads).sqrt()
        norm = T.grad_norm(grads)
        assert abs(float(norm) - float(norm64)) <= 34 * 2.0 ** -24 * float(norm64), (scale, odd)
        before = [g.double() for g in grads]
        bound = 0.5 * float(norm64)
        assert torch.equal(T.clip_grads(grads, bound), norm)
        factor = bound / (float(norm64) + 1e-6)
        for g, b in zip(grads, before):
            within(g, b * factor, 38 * 2.0 ** -24 * (b * factor).abs() + 2.0 ** -149)
    for odd in (float("inf"), float("nan")):
        grads = [draw(1, n, "f32", i)[0] for i in range(count)]
        grads[-1][-1] = odd
        got = float(T.clip_grads(grads, 1.0))
        assert got == odd or (odd != odd and got != got)
        assert bool(grads[0][:-1].isnan().all() if odd != odd else (grads[0][:-1] == 0).all())
