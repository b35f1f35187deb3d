"""GPU parity of the layer norm and its gradients with the float64 definitions.

Tolerances, from the kernels' arithmetic (fp32, one rounding to the output's
type, half a spacing):
  - h is one fp32 addition and one rounding;
  - a sum over a row adds at most (terms a thread + 10 tree levels) times, under
    64 for rows up to 40000 columns (5 vectors of 8 a thread): its error is at
    most 2^-18 of the sum of magnitudes;
  - d = h - m rounds h (2^-24 |h|) and itself (2^-24 |d|), and is corrected by
    its mean, which is off by 2^-18 of the mean of |d|; the same holds of what
    the correction itself rounds, so d is within
    2^-23 |h| + 2^-22 |d| + 2^-18 mean|d|;
  - the variance, a sum of squares of such d, is within 2^-17 of itself plus
    twice what the errors 2^-23 |h| make of the d, rstd within half of that.
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

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SHAPES = [(1, 4096), (3, 1), (5, 7), (33, 128), (17, 200), (4, 129), (2, 3000), (9, 4104),
          (2, 8200), (2, 16500), (2, 40000), (700, 256), (1, 64), (400, 1024), (330, 4001)]


def draw(shape, dtype, seed, scale=1.0, mean=0.0, pitch=None, shift=0):
    """Normals of a type about a mean, as a view with a row pitch and an offset."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols = shape
    pitch = pitch or cols
    full = torch.randn(rows * pitch + shift, generator=g, device="cuda") * scale + mean
    return full.to(DT[dtype])[shift:].view(rows, pitch)[:, :cols]


def f64(t):
    return t.double().cpu().numpy()


def within(got, ref, slack, dtype):
    err = np.abs(f64(got) - ref)
    tol = OT.ulp(ref, dtype) / 2 * (1 + 2.0 ** -6) + slack
    assert np.all(err <= tol), f"worst error/tolerance {np.max(err / tol)}"


def norm_slack(h, w, b, eps):
    """What y may be off by before its rounding."""
    d = h - h.mean(1, keepdims=True)
    md = np.abs(d).mean(1, keepdims=True)
    mh = np.abs(h).mean(1, keepdims=True)
    var = (d * d).mean(1, keepdims=True)
    r = 1 / np.sqrt(var + eps)
    off = 2.0 ** -23 * np.abs(h) + 2.0 ** -22 * np.abs(d) + 2.0 ** -18 * md
    rel = 2.0 ** -18 + (2.0 ** -23 * mh * md + 2.0 ** -46 * mh * mh) * r * r
    n = np.abs(d) * r * np.abs(w)
    return off * r * np.abs(w) + n * rel + 2.0 ** -22 * (n + np.abs(b))


def check_norm(x, w, b, r, eps=1e-5, y=None, **kw):
    dtype = {v: k for k, v in DT.items()}[x.dtype]
    x64, w64 = f64(x), f64(w)
    b64 = np.zeros_like(w64) if b is None else f64(b)
    y64, h64 = OO.layernorm(x64, w64, b64, None if r is None else f64(r), eps)
    got, h = T.layernorm(x, w, b, residual=r, eps=eps, **kw) if y is None else y
    slack = norm_slack(h64, w64, b64, eps)
    within(got, y64, slack, dtype)
    if r is not None:
        within(h, h64, 2.0 ** -24 * np.abs(h64), dtype)
    return y64, slack


def check_fp8(q, scales, y64, slack):
    s = f64(scales)
    want = OO.row_scales(y64)
    most = OO.row_scales(np.abs(y64) + slack) - want      # slack at the block's largest
    assert s.shape == want.shape
    assert np.all(np.abs(s - want) <= most + 2.0 ** -22 * want)
    sp = OO.spread(s, y64.shape[1], 1)
    # The quotient is within two units of fp32's; y / scale may reach a little over 448.
    err = np.abs(f64(q) * sp - y64)
    top = OO.spread(most, y64.shape[1], 1) * 448
    assert np.all(err <= sp * OO.half_step(y64 / sp) * (1 + 2 ** -8) + slack + top +
                  2.0 ** -21 * np.abs(y64))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("residual,bias", [(False, True), (True, True), (True, False)])
def test_norm_all_outputs(shape, dtype, residual, bias):
    x = draw(shape, dtype, 1, mean=0.5)
    r = draw(shape, dtype, 2, mean=-1.0) if residual else None
    w = draw((1, shape[1]), dtype, 3)[0]
    b = draw((1, shape[1]), dtype, 4)[0] if bias else None
    y64, slack = check_norm(x, w, b, r)
    q, s, h = T.layernorm_fp8(x, w, b, residual=r)
    check_fp8(q, s, y64, slack)
    if not residual:
        assert h is x
    else:
        assert torch.equal(h, T.layernorm(x, w, b, residual=r)[1])


@pytest.mark.parametrize("shift,pitch", [(0, 136), (1, 131), (8, 160), (4, 130)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_strided_and_unaligned_rows(shift, pitch, dtype):
    shape = (6, 128)
    x, r = draw(shape, dtype, 4, pitch=pitch, shift=shift), draw(shape, dtype, 5)
    w, b = draw((1, 128), "f32", 6)[0], draw((1, 128), "f32", 7)[0]
    full = torch.full((6, pitch), 7.0, dtype=DT[dtype], device="cuda")
    y64, slack = check_norm(x, w, b, r, out=full[:, :128])
    assert bool((full[:, 128:] == 7.0).all())
    q, s, _ = T.layernorm_fp8(x, w, b, residual=r,
                              scales=torch.empty((6, 3), device="cuda")[:, 1:2])
    check_fp8(q, s, y64, slack)


@pytest.mark.parametrize("shape", [(5, 300), (5, 40000), (400, 2048)], ids=str)
def test_norm_in_place(shape):
    x, r = draw(shape, "bf16", 7), draw(shape, "bf16", 8)
    w = draw((1, shape[1]), "bf16", 9)[0]
    y_ref, h_ref = T.layernorm(x, w, residual=r)
    y, h = T.layernorm(x, w, residual=r, h_out=r)
    assert h is r and torch.equal(h, h_ref) and torch.equal(y, y_ref)
    # Without a residual h is a copy.
    hh = torch.empty_like(x)
    _, h = T.layernorm(x, w, h_out=hh)
    assert h is hh and torch.equal(hh, x)


@pytest.mark.parametrize("shape", [(3, 4096), (400, 4096), (3, 33), (3, 40000)], ids=str)
@pytest.mark.parametrize("mean", [1e3, -3e5])
def test_rows_far_from_zero_keep_their_spread(shape, mean):
    # The mean of 4096 fp32 numbers at 3e5 is good to 0.02 or so; y must be too,
    # but as far as the numbers themselves are: they are exact here.
    x = draw(shape, "f32", 10, mean=mean)
    w = draw((1, shape[1]), "f32", 11)[0]
    check_norm(x, w, None, None)


def test_norm_of_constant_rows_zeros_infinities_and_nans():
    w, b = draw((1, 256), "f32", 12)[0], draw((1, 256), "f32", 13)[0]
    for rows in (6, 500):                                # few rows and many
        x = draw((rows, 256), "f32", 14)
        x[0] = 0.0
        x[1] = 3.0
        x[2, 17] = float("inf")
        x[3, 200] = float("nan")
        y, _ = T.layernorm(x, w, b)
        assert torch.equal(y[0], b) and torch.equal(y[1], b)
        assert bool(y[2:4].isnan().all()) and bool(y[4:].isfinite().all())
        q, s, _ = T.layernorm_fp8(x, w, b)
        assert bool(s[2:4].isnan().all()) and bool(q[2:4].float().isnan().all())
        assert bool(s[[0, 1, 4, 5]].isfinite().all())
        zero = torch.zeros_like(b)
        q, s, _ = T.layernorm_fp8(x[:2], w, zero)
        assert bool((q.float() == 0).all()) and bool((s == 2.0 ** -126).all())


def test_no_rows():
    x, w = torch.empty((0, 64), device="cuda"), torch.ones(64, device="cuda")
    y, h = T.layernorm(x, w)
    assert y.shape == (0, 64) and h is x
    dx, dw, db = T.layernorm_grad(x, x, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


# ---- gradients --------------------------------------------------------------------------


def check_grad(dy, h, w, dh, eps=1e-5, got=None):
    dtype = {v: k for k, v in DT.items()}[h.dtype]
    dy64, h64, w64 = f64(dy), f64(h), f64(w)
    dh64 = None if dh is None else f64(dh)
    rx, rw, rb = OO.layernorm_grad(dy64, h64, w64, dh64, eps)
    dx, dw, db = got or T.layernorm_grad(dy, h, w, eps=eps, dh=dh)
    d = h64 - h64.mean(1, keepdims=True)
    md = np.abs(d).mean(1, keepdims=True)
    u = (d * d).mean(1, keepdims=True) + eps
    r = 1 / np.sqrt(u)
    g = np.abs(dy64 * w64)
    mg = g.mean(1, keepdims=True)
    # Errors of d as above (h itself is exact), of the sums 2^-18 of magnitudes.
    off = 2.0 ** -22 * np.abs(d) + 2.0 ** -18 * md
    mgd = (g * np.abs(d)).mean(1, keepdims=True) + 2.0 ** -18 * mg * md
    slack = 2.0 ** -17 * (g * r + mg * r + np.abs(d) * mgd * r ** 3) + off * mgd * r ** 3
    slack += (np.abs(d) + off) * (mg * 2.0 ** -17 * md) * r ** 3
    if dh is not None:
        slack += 2.0 ** -23 * np.abs(dh64)
    within(dx, rx, slack, dtype)
    # A column's terms go through at most rows / 64 additions in a block and a
    # tree; every term is off by what d and rstd are.
    chain = (h64.shape[0] / 64 + 40) * 2.0 ** -24
    each = np.abs(dy64) * np.abs(d) * r
    within(dw, rw, each.sum(0) * (chain + 2.0 ** -17) + (np.abs(dy64) * off * r).sum(0), "f32")
    within(db, rb, np.abs(dy64).sum(0) * chain, "f32")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES + [(3000, 520), (2500, 72)], ids=str)
@pytest.mark.parametrize("past", [False, True])
def test_gradients(shape, dtype, past):
    dy, h = draw(shape, dtype, 21), draw(shape, dtype, 22, mean=0.7)
    w = draw((1, shape[1]), "f32" if past else dtype, 23)[0]
    check_grad(dy, h, w, draw(shape, dtype, 24) if past else None)


@pytest.mark.parametrize("shift,pitch", [(1, 131), (8, 160), (4, 130)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_strided_rows(shift, pitch, dtype):
    shape = (700, 128)
    dy, h = draw(shape, dtype, 25, pitch=pitch, shift=shift), draw(shape, dtype, 26)
    w, dh = draw((1, 128), "f16", 27)[0], draw(shape, dtype, 28, pitch=pitch)
    full = torch.full((700, pitch), 7.0, dtype=DT[dtype], device="cuda")
    sums = torch.full((3, 128), 7.0, device="cuda")
    got = T.layernorm_grad(dy, h, w, dh=dh, dx_out=full[:, :128], dweight_out=sums[0],
                           dbias_out=sums[2])
    check_grad(dy, h, w, dh, got=got)
    assert bool((full[:, 128:] == 7.0).all()) and bool((sums[1] == 7.0).all())


def test_gradient_against_differences_of_the_norm():
    # The kernel's gradient against central differences of the definition in 64 bits.
    rng = np.random.default_rng(3)
    x, dy, w = rng.normal(size=(2, 40)), rng.normal(size=(2, 40)), rng.normal(size=40)
    dx, dw, db = T.layernorm_grad(*(torch.tensor(t, device="cuda", dtype=torch.float32)
                                    for t in (dy, x, w)))
    x, dy, w = (np.float64(np.float32(t)) for t in (x, dy, w))

    def loss(x, w):
        return (OO.layernorm(x, w)[0] * dy).sum()

    step = 1e-5
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = step
        num = (loss(x + e, w) - loss(x - e, w)) / (2 * step)
        assert abs(num - float(dx[i])) < 2e-6 * (1 + np.abs(dy * w).max())
    for j in range(40):
        e = np.zeros_like(w)
        e[j] = step
        num = (loss(x, w + e) - loss(x, w - e)) / (2 * step)
        assert abs(num - float(dw[j])) < 2e-6 * (1 + np.abs(dy).sum())


def test_gradients_are_the_same_every_time_and_far_rows_are_right():
    dy, h = draw((5000, 3000), "bf16", 30), draw((5000, 3000), "bf16", 31, mean=2.0)
    w = draw((1, 3000), "bf16", 32)[0]
    first = T.layernorm_grad(dy, h, w)
    ws = T.layernorm_grad_workspace(h)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, T.layernorm_grad(dy, h, w, workspace=ws)))
    h = draw((50, 1000), "f32", 33, mean=1e4)
    check_grad(draw((50, 1000), "f32", 34), h, draw((1, 1000), "f32", 35)[0], None)


def test_a_workspace_that_is_too_small_is_refused():
    dy = draw((400, 64), "bf16", 36)
    with pytest.raises(T.TilesError, match="workspace"):
        T.layernorm_grad(dy, dy, dy[0], workspace=T.workspace())
