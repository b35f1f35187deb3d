"""GPU parity of the norm, its gradients and the block quantiser with the
float64 definitions.

Tolerances, from the kernels' arithmetic (fp32 throughout, one rounding to
the output type):
  - a row's sum of squares adds non-negative terms: its relative error is at
    most (terms a thread + 10 tree levels) * 2^-24, under 2^-18 for rows up to
    40000 columns (5 vectors of 8 a thread); rstd halves it.  A 16-bit or fp32
    y is then within 2^-18 of itself plus one spacing of its type;
  - h is one fp32 addition and one rounding;
  - gradients: the same relative error on the sum of the magnitudes;
    dweight adds up to 16384 rows in blocks: 2^-14 of the magnitudes' sum
    covers a chain of 1000 fp32 additions;
  - an 8-bit value is within half a spacing of y / scale, and a scale within
    2^-18 of the largest magnitude over 448.
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
REL = 2.0 ** -18
SHAPES = [(1, 4096), (3, 1), (5, 7), (33, 128), (17, 200), (4, 129), (2, 3000), (9, 4104),
          (2, 8200), (2, 16500), (2, 40000), (700, 256), (1, 64)]


def draw(shape, dtype, seed, scale=1.0, pitch=None, shift=0):
    """Normals of a type, as a view with a row pitch and an offset of its own."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols = shape
    pitch = pitch or cols
    full = torch.randn(rows * pitch + shift, generator=g, device="cuda") * scale
    return full.to(DT[dtype])[shift:].view(rows, pitch)[:, :cols]


def f64(t):
    return t.double().cpu().numpy()


def assert_within(got, ref, bound, dtype, rel=REL):
    ok, worst, idx = OT.check(f64(got), ref, bound, dtype, rel)
    assert ok, f"worst error/tolerance {worst} at {idx}"


def assert_fp8(q, scales, y64):
    s = f64(scales)
    want = OO.row_scales(y64)
    assert s.shape == want.shape
    assert np.all(np.abs(s - want) <= REL * want)
    sp = OO.spread(s, y64.shape[1], 1)
    # y / scale reaches 448 * (1 + REL) at most, which saturates.
    err = np.abs(f64(q) * sp - y64)
    assert np.all(err <= sp * OO.half_step(y64 / sp) * (1 + 2 ** -8) + REL * np.abs(y64))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_all_outputs(shape, dtype, residual):
    x = draw(shape, dtype, 1)
    r = draw(shape, dtype, 2) if residual else None
    w = draw((1, shape[1]), dtype, 3)[0]
    y64, h64 = OO.rmsnorm(f64(x), f64(w), f64(r) if residual else None)
    y, h = T.rmsnorm(x, w, residual=r)
    assert_within(y, y64, np.abs(y64), dtype)
    q, s, h8 = T.rmsnorm_fp8(x, w, residual=r)
    assert_fp8(q, s, y64)
    if residual:
        assert_within(h, h64, np.abs(h64), dtype, 2.0 ** -24)
        assert torch.equal(h, h8)
    else:
        assert h is x and h8 is x


@pytest.mark.parametrize("shift,pitch", [(0, 136), (1, 131), (8, 160), (4, 130)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_strided_and_unaligned_rows(shift, pitch, dtype):
    shape = (6, 128)
    x, r = draw(shape, dtype, 4, pitch=pitch, shift=shift), draw(shape, dtype, 5)
    w = draw((1, 128), "f32", 6)[0]
    y64, h64 = OO.rmsnorm(f64(x), f64(w), f64(r))
    full = torch.full((6, pitch), 7.0, dtype=DT[dtype], device="cuda")
    y, h = T.rmsnorm(x, w, residual=r, out=full[:, :128])
    assert_within(y, y64, np.abs(y64), dtype)
    assert bool((full[:, 128:] == 7.0).all())
    q, s, _ = T.rmsnorm_fp8(x, w, residual=r,
                            scales=torch.empty((6, 3), device="cuda")[:, 1:2])
    assert_fp8(q, s, y64)


def test_norm_updates_the_residual_in_place():
    x, r = draw((5, 40000), "bf16", 7), draw((5, 40000), "bf16", 8)
    w = draw((1, 40000), "bf16", 9)[0]
    y_ref, h_ref = T.rmsnorm(x, w, residual=r)
    y, h = T.rmsnorm(x, w, residual=r, h_out=r)
    assert h is r and torch.equal(h, h_ref) and torch.equal(y, y_ref)


def test_norm_of_zeros_infinities_and_nans():
    x = draw((5, 300), "bf16", 10)
    x[0] = 0
    x[1, 7] = float("nan")
    x[2, 299] = float("inf")
    x[3] *= 1e-30
    w = torch.ones(300, dtype=torch.bfloat16, device="cuda")
    y, _ = T.rmsnorm(x, w)
    h32 = x.float()
    want = h32 * torch.rsqrt((h32 * h32).mean(1, keepdim=True) + 1e-6)
    assert torch.equal(y.isnan(), want.bfloat16().isnan())
    assert bool((y[0] == 0).all()) and bool((y[2, :299] == 0).all())
    q, s, _ = T.rmsnorm_fp8(x, w)
    assert bool((q[0].float() == 0).all()) and bool((s[0] == OO.TINY_SCALE).all())
    assert bool(s[1].isnan().all()) and bool(q[1].float().isnan().all())
    # Row 2: y is zero but for a NaN at the infinity, in the last block.
    assert bool(s[2, 2].isnan()) and bool((s[2, :2] == OO.TINY_SCALE).all())
    y64, _ = OO.rmsnorm(f64(x[3:]), f64(w))
    assert_fp8(q[3:], s[3:], y64)


@pytest.mark.parametrize("rows,cols", [(4, 512), (700, 512), (700, 1024)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_quiet_rows_with_blocks_of_zeros(rows, cols, residual):
    # 1 / sqrt(mean + eps) is 1000 here and a block of zeros has the smallest
    # scale: their quotient is past fp32, the values are not.
    x = draw((rows, cols), "bf16", 13, 1e-4)
    x[:, 128:256] = 0
    x[1] = 0
    x[2, :128] = 2.0 ** -130
    r = torch.zeros_like(x) if residual else None
    w = draw((1, cols), "bf16", 14)[0]
    q, s, _ = T.rmsnorm_fp8(x, w, residual=r)
    y64, _ = OO.rmsnorm(f64(x), f64(w))
    assert bool((q[:, 128:256].float() == 0).all()) and bool((s[:, 1] == OO.TINY_SCALE).all())
    assert bool(q.float().isfinite().all())
    assert_fp8(q, s, y64)


def test_norm_of_no_rows_and_of_another_stream():
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    y, h = T.rmsnorm(torch.empty((0, 64), dtype=torch.float16, device="cuda"), w)
    assert y.shape == (0, 64)
    q, s, _ = T.rmsnorm_fp8(torch.empty((0, 64), dtype=torch.float16, device="cuda"), w)
    assert q.shape == (0, 64) and s.shape == (0, 1)
    side = torch.cuda.Stream()
    x = draw((2000, 2048), "f16", 11)
    w = draw((1, 2048), "f16", 12)[0]
    want, _ = T.rmsnorm(x, w)
    side.wait_stream(torch.cuda.current_stream())
    got, _ = T.rmsnorm(x, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES + [(5000, 96), (1500, 1024)], ids=str)
@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_gradients(shape, dtype, with_dh):
    h, dy = draw(shape, dtype, 20), draw(shape, dtype, 21)
    dh = draw(shape, dtype, 22) if with_dh else None
    w = draw((1, shape[1]), dtype, 23)[0]
    ws = T.rmsnorm_grad_workspace(h)
    dx, dw = T.rmsnorm_grad(dy, h, w, dh=dh, workspace=ws)
    rx, rw, bx, bw = OO.rmsnorm_grad(f64(dy), f64(h), f64(w), f64(dh) if with_dh else None)
    assert_within(dx, rx, bx, dtype)
    assert_within(dw, rw, bw, "f32", 2.0 ** -14)
    again = T.rmsnorm_grad(dy, h, w, dh=dh, workspace=ws)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_norm_gradients_against_differences():
    # fp32 rows: the loss sum(y * dy) + sum(h * dh) in float64 at h +- step e.
    h, dy, dh = (draw((4, 40), "f32", s) for s in (24, 25, 26))
    w = draw((1, 40), "f32", 27)[0]
    dx, dw = T.rmsnorm_grad(dy, h, w, eps=1e-3, dh=dh, workspace=T.rmsnorm_grad_workspace(h))
    h64, dy64, dh64, w64 = f64(h), f64(dy), f64(dh), f64(w)

    def loss(h_, w_):
        y, _ = OO.rmsnorm(h_, w_, eps=1e-3)
        return (y * dy64).sum() + (h_ * dh64).sum()

    step = 1e-5
    for i, j in [(0, 0), (1, 17), (3, 39)]:
        d = np.zeros_like(h64)
        d[i, j] = step
        num = (loss(h64 + d, w64) - loss(h64 - d, w64)) / (2 * step)
        assert abs(num - float(dx[i, j])) < 1e-4
    d = np.zeros_like(w64)
    d[5] = step
    assert abs((loss(h64, w64 + d) - loss(h64, w64 - d)) / (2 * step) - float(dw[5])) < 1e-4


def test_norm_gradient_of_strided_rows_and_no_rows():
    h, dy = draw((9, 130), "bf16", 28, pitch=133, shift=1), draw((9, 130), "bf16", 29, pitch=136)
    w = draw((1, 130), "f32", 30)[0]
    dx, dw = T.rmsnorm_grad(dy, h, w, workspace=T.rmsnorm_grad_workspace(h))
    rx, rw, bx, bw = OO.rmsnorm_grad(f64(dy), f64(h), f64(w))
    assert_within(dx, rx, bx, "bf16")
    assert_within(dw, rw, bw, "f32", 2.0 ** -14)
    none = torch.empty((0, 130), dtype=torch.bfloat16, device="cuda")
    dx, dw = T.rmsnorm_grad(none, none, w, workspace=T.rmsnorm_grad_workspace(none))
    assert dx.shape == (0, 130) and bool((dw == 0).all())


def test_norm_gradient_refuses_a_small_workspace():
    h = draw((600, 512), "bf16", 31)
    w = draw((1, 512), "bf16", 32)[0]
    with pytest.raises(T.TilesError):
        T.rmsnorm_grad(h, h, w)
    with pytest.raises(T.TilesError):
        T.rmsnorm_grad(h, h, w, workspace=T.rmsnorm_grad_workspace(h)[:-4])


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 128), (130, 257), (128, 384), (5, 4100), (2, 200, 136),
                                   (3, 1, 77)], ids=str)
def test_quantise_rows_and_blocks(shape, dtype):
    lead, rows, cols = (1, *shape) if len(shape) == 2 else shape
    x = torch.stack([draw((rows, cols), dtype, 40 + i, 10.0 ** i) for i in range(lead)])
    x = x.view(shape)
    q, s = T.quantize_fp8(x)
    qb, sb = T.quantize_fp8(x, block_rows=128)
    for i in range(lead):
        one = (lambda t: t[i]) if len(shape) == 3 else (lambda t: t)
        x64 = f64(one(x))
        assert_fp8(one(q), one(s), x64)
        want = OO.square_scales(x64)
        got = f64(one(sb))
        assert np.all(np.abs(got - want) <= REL * want)
        sp = OO.spread(OO.spread(got, cols, 1), rows, 0)
        err = np.abs(f64(one(qb)) * sp - x64)
        assert np.all(err <= sp * OO.half_step(x64 / sp) * (1 + 2 ** -8) + REL * np.abs(x64))
    assert q.stride(-2) % 16 == 0 and qb.stride(-2) % 16 == 0


def test_quantise_zeros_and_nans():
    x = torch.zeros((130, 130), dtype=torch.float16, device="cuda")
    x[129, 3] = float("nan")
    q, s = T.quantize_fp8(x)
    assert bool(s[129, 0].isnan()) and bool((s[:129] == OO.TINY_SCALE).all())
    assert bool((q[:129].float() == 0).all()) and bool(q[129, 3].float().isnan())
    q, s = T.quantize_fp8(x, block_rows=128)
    assert bool(s[1, 0].isnan()) and bool((s[0] == OO.TINY_SCALE).all())


def test_python_refusals():
    x = draw((4, 64), "bf16", 50)
    w = draw((1, 64), "bf16", 51)[0]
    with pytest.raises(ValueError):
        T.rmsnorm(x, w[:32])
    with pytest.raises(ValueError):
        T.rmsnorm(x.t(), w)
    with pytest.raises(ValueError):
        T.rmsnorm(x.cpu(), w)
    with pytest.raises(TypeError):
        T.rmsnorm(x, w, residual=x.float())
    with pytest.raises(ValueError):
        T.rmsnorm_fp8(x, w, scales=torch.empty((4, 2), device="cuda"))
    with pytest.raises(ValueError):
        T.quantize_fp8(x, block_rows=64)
    with pytest.raises(TypeError):
        T.rmsnorm(x.double(), w)
