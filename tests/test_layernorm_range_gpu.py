"""GPU tests of the layer norm and its gradients where the squares of a row's deviations
leave fp32's range although the row is finite: such a row is NaN and no other row is
touched; one whose squares' sum fp32 still holds is as right as any.

Tolerances: of a row within the range as in the tests of many rows, 2^-17 of the
magnitudes that enter and half a spacing of the output's type (2^-8, 2^-11 or 2^-24 of
the value); the 8-bit values half a step (2^-4) more, their scales 2^-17."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}

# Rows whose threads hold one, two or four vectors of them, or none (any length); few
# rows and many, whose kernels keep the next rows on their way in; rows off 16 bytes.
SHAPES = [(6, 96), (6, 304), (6, 301), (5, 9000), (5, 20000), (5, 20001), (5, 40000), (1300, 1024),
          (3000, 1001), (700, 3200)]
OVER, SUM, UNDER = 1, 2, 3                     # the rows that matter


def matrix(rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x[OVER] *= 1e20                            # squares past the range
    x[SUM] = 1.5e19 * x[SUM].sign()            # squares within, not their sum
    x[UNDER] *= 1e16
    return x.to(dtype)


def draw(*shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def rest(rows):
    return [i for i in range(rows) if i not in (OVER, SUM)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_a_finite_row_whose_squares_leave_the_range(rows, cols, residual, dtype):
    x, w, b = matrix(rows, cols, dtype), draw(cols, dtype=dtype, seed=2), draw(cols, dtype=dtype, seed=3)
    assert bool(x.isfinite().all())
    r = torch.zeros_like(x) if residual else None
    y, _ = T.layernorm(x, w, b, residual=r)
    q, s, _ = T.layernorm_fp8(x, w, b, residual=r)
    for i in (OVER, SUM):
        assert bool(y[i].isnan().all()) and bool(s[i].isnan().all()) and bool(q[i].float().isnan().all())
    keep = rest(rows)
    h = x[keep].double()
    d = h - h.mean(1, keepdim=True)
    rstd = ((d * d).mean(1, keepdim=True) + 1e-5).rsqrt()
    want = d * rstd * w.double() + b.double()
    size = (d.abs() + d.abs().mean(1, keepdim=True) + 2.0 ** -6 * h.abs()) * rstd * w.double().abs() + b.double().abs()
    tol = want.abs() * HALF[dtype] + 2.0 ** -17 * size
    assert bool(((y[keep].double() - want).abs() <= tol).all())
    spread = s[keep].double().repeat_interleave(128, 1)[:, :cols]
    err = (q[keep].double() * spread - want).abs()
    assert bool((err <= want.abs() * 2.0 ** -4 + spread * 2.0 ** -10 + 2.0 ** -16 * size).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("past", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_the_gradients_of_such_a_row(rows, cols, past, dtype):
    h, w, dy = matrix(rows, cols, dtype), draw(cols, dtype=dtype, seed=2), draw(rows, cols, dtype=dtype, seed=4)
    dh = draw(rows, cols, dtype=dtype, seed=5) if past else None
    dx, dw, db = T.layernorm_grad(dy, h, w, dh=dh)
    assert bool(dx[OVER].isnan().all()) and bool(dx[SUM].isnan().all()) and bool(dw.isnan().all())
    keep = rest(rows)
    assert bool(dx[keep].isfinite().all()) and bool(db.isfinite().all())
    # The same rows without the two others among them; all finite.
    clean = h.clone()
    clean[[OVER, SUM]] = h[[0, 0]]
    cx, cw, cb = T.layernorm_grad(dy, clean, w, dh=dh)
    assert torch.equal(cx[keep], dx[keep]) and torch.equal(cb, db) and bool(cw.isfinite().all())
    v = clean.double()
    d = v - v.mean(1, keepdim=True)
    r = ((d * d).mean(1, keepdim=True) + 1e-5).rsqrt()
    g = dy.double() * w.double()
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    want = (g - mean(g)) * r - d * mean(g * d) * r ** 3
    size = (g.abs() + mean(g.abs())) * r + d.abs() * mean((g * d).abs()) * r ** 3 + d.abs() * mean(g.abs()) * r * r
    if past:
        want, size = want + dh.double(), size + dh.double().abs()
    tol = want.abs() * HALF[dtype] + 2.0 ** -17 * size
    assert bool(((cx.double() - want).abs() <= tol).all())
