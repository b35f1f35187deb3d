"""GPU parity of the norm's kernel for many long 16-bit rows, whose blocks take
several rows in turn: every output against the float64 definition, at the
tolerances of test_norm_gpu (derived there), and through the C call where the
Python one does not go."""

import ctypes as C

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
CODE = {"f16": _abi.F16, "bf16": _abi.BF16, "f32": _abi.F32}


def draw(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(DT[dtype])


def c_norm(x, w, residual, h, fp8, dtype):
    """tiles_rmsnorm with every pointer as given; (y, scales)."""
    rows, cols = x.shape
    y = torch.empty((rows, cols), dtype=torch.float8_e4m3fn if fp8 else DT[dtype], device="cuda")
    s = torch.empty((rows, OO.blocks(cols)), device="cuda")
    d = _abi.RmsnormDesc(rows=rows, cols=cols, x=x.data_ptr(), weight=w.data_ptr(),
                         residual=residual.data_ptr() if residual is not None else None,
                         h=h.data_ptr() if h is not None else None, y=y.data_ptr(),
                         scales=s.data_ptr() if fp8 else None, ldx=x.stride(0), ldr=cols,
                         ldh=h.stride(0) if h is not None else 0, ldy=cols,
                         scale_row=OO.blocks(cols), scale_block=1, eps=1e-6, dtype=CODE[dtype],
                         weight_dtype=CODE[dtype], out_dtype=_abi.E4M3 if fp8 else CODE[dtype])
    stream = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert T.load().tiles_rmsnorm(C.byref(d), stream) == _abi.OK
    return y, s


# Few rows and many, rows that start on 16 bytes and rows that do not, 16 bits
# and 32: every kernel that may run.
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(3, 1024), (700, 1024), (700, 1001), (700, 8192), (400, 256),
                                       (2, 40000)])
@pytest.mark.parametrize("fp8", [False, True])
def test_h_without_a_residual_is_x(rows, cols, dtype, fp8):
    x, w = draw((rows, cols), dtype, 1), draw((cols,), dtype, 2)
    want, ws = c_norm(x, w, None, None, fp8, dtype)
    h = torch.full((rows, cols + 8), 7.0, dtype=DT[dtype], device="cuda")
    y, s = c_norm(x, w, None, h[:, :cols], fp8, dtype)
    assert torch.equal(h[:, :cols], x) and bool((h[:, cols:] == 7.0).all())
    assert torch.equal(y.view(torch.uint8), want.view(torch.uint8))
    assert not fp8 or torch.equal(s, ws)


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("norm", ["rmsnorm", "rmsnorm_fp8"])
def test_h_out_without_a_residual_is_written(norm, compiled, monkeypatch):
    T._compiled()
    if not compiled:
        monkeypatch.setattr(T, "_CALLS", T._NoCalls)
    x, w = draw((5, 304), "bf16", 3), draw((304,), "bf16", 4)
    out = torch.full((5, 320), 7.0, dtype=torch.bfloat16, device="cuda")
    view = out[:, :304]
    h = getattr(T, norm)(x, w, h_out=view)[-1]
    assert h is view and torch.equal(h, x) and bool((out[:, 304:] == 7.0).all())
    assert getattr(T, norm)(x, w)[-1] is x
    with pytest.raises((ValueError, TypeError)):
        getattr(T, norm)(x, w, h_out=out)
    with pytest.raises((ValueError, TypeError)):
        getattr(T, norm)(x, w, h_out=view.half())


def assert_norm(x, w, r, eps, fp8):
    """At the tolerances of test_norm_gpu: 2^-18 of y and one spacing of its
    type; half an 8-bit step and 2^-18; scales within 2^-18."""
    f64 = lambda t: t.double().cpu().numpy()
    rel = 2.0 ** -18
    y64, h64 = OO.rmsnorm(f64(x), f64(w), f64(r) if r is not None else None, eps)
    if fp8:
        q, s, h = T.rmsnorm_fp8(x, w, residual=r, eps=eps)
        want, s = OO.row_scales(y64), f64(s)
        assert np.all(np.abs(s - want) <= rel * want)
        sp = OO.spread(s, y64.shape[1], 1)
        err = np.abs(f64(q) * sp - y64)
        assert np.all(err <= sp * OO.half_step(y64 / sp) * (1 + 2 ** -8) + rel * np.abs(y64))
    else:
        y, h = T.rmsnorm(x, w, residual=r, eps=eps)
        name = {v: k for k, v in DT.items()}[x.dtype]
        ok, worst, idx = OT.check(f64(y), y64, np.abs(y64), name, rel)
        assert ok, (worst, idx)
    if r is not None:
        ok, worst, idx = OT.check(f64(h), h64, np.abs(h64), {v: k for k, v in DT.items()}[h.dtype],
                                  2.0 ** -24)
        assert ok, (worst, idx)


# h * weight leaves fp32's range on either side, the norm's output does not.
@pytest.mark.parametrize("rows,cols", [(5, 1024), (700, 1024), (700, 2056), (350, 8192)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("hscale,wscale,eps", [(2.0 ** 20, 2.0 ** 118, 1e-6),
                                               (2.0 ** -45, 2.0 ** -100, 0.0)])
def test_norm_whose_products_leave_the_range(rows, cols, fp8, residual, hscale, wscale, eps):
    # Powers of two: the oracle's inputs are the kernel's.  One block of 128
    # columns keeps an ordinary weight, one is zero.
    x = (draw((rows, cols), "f32", 5) * hscale).bfloat16()
    r = (draw((rows, cols), "f32", 6) * hscale).bfloat16() if residual else None
    w = draw((cols,), "f32", 7)
    w = torch.where(w.abs() < 0.1, torch.ones_like(w), w) * wscale
    w[256:384] /= wscale
    x[:, 512:640] = 0
    if residual:
        r[:, 512:640] = 0
    assert_norm(x, w, r, eps, fp8)


# Blocks with one row and with dozens, rows of whole and of short last blocks of
# 128; the last is past 160 MB with a residual (fewer blocks an SM).
SHAPES = [(305, 520), (700, 1024), (400, 3000), (350, 8192), (12000, 1032), (6000, 4104)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_every_output(shape, dtype, residual, fp8):
    x, w = draw(shape, dtype, 11), draw((shape[1],), dtype, 12)
    r = draw(shape, dtype, 13) if residual else None
    assert_norm(x, w, r, 1e-6, fp8)


@pytest.mark.parametrize("shape", [(700, 1024), (12000, 1032), (6000, 4104)], ids=str)
@pytest.mark.parametrize("over", ["residual", "x"])
@pytest.mark.parametrize("fp8", [False, True])
def test_h_over_its_input(shape, over, fp8):
    x, r, w = draw(shape, "bf16", 14), draw(shape, "bf16", 15), draw((shape[1],), "f32", 16)
    norm = T.rmsnorm_fp8 if fp8 else T.rmsnorm
    want = norm(x, w, residual=r)
    target = r if over == "residual" else x
    got = norm(x, w, residual=r, h_out=target)
    assert got[-1] is target and torch.equal(target, want[-1])
    for u, v in zip(got[:-1], want[:-1]):
        assert torch.equal(u.view(torch.uint8) if fp8 and u.element_size() == 1 else u,
                           v.view(torch.uint8) if fp8 and v.element_size() == 1 else v)


@pytest.mark.parametrize("shift,pitch", [(0, 1040), (8, 1048), (0, 2048)])
def test_rows_with_a_pitch_keep_what_lies_between(shift, pitch):
    rows, cols = 2000, 1032
    full = draw((rows * pitch + shift,), "bf16", 17)
    x = full[shift:].view(rows, pitch)[:, :cols]
    w = draw((cols,), "bf16", 18)
    out = torch.full((rows, pitch), 7.0, dtype=torch.bfloat16, device="cuda")
    h = torch.full((rows, pitch), 7.0, dtype=torch.bfloat16, device="cuda")
    want = T.rmsnorm(x.contiguous(), w, residual=x.contiguous())
    got = T.rmsnorm(x, w, residual=x, out=out[:, :cols], h_out=h[:, :cols])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((out[:, cols:] == 7.0).all()) and bool((h[:, cols:] == 7.0).all())


def test_nans_and_infinities_stay_in_their_rows():
    x, w = draw((2000, 1032), "f16", 19), torch.ones(1032, dtype=torch.float16, device="cuda")
    plain = T.rmsnorm_fp8(x, w)
    want = [plain[0].float(), plain[1].clone()]
    x[7, 5], x[900, 1031], x[1999, 0] = float("nan"), float("inf"), float("-inf")
    q, s, _ = T.rmsnorm_fp8(x, w)
    q = q.float()
    keep = torch.ones(2000, dtype=torch.bool)
    keep[[7, 900, 1999]] = False
    assert torch.equal(q[keep], want[0][keep]) and torch.equal(s[keep], want[1][keep])
    assert bool(q[7].isnan().all()) and bool(s[7].isnan().all())
    # h / rms is zero but for inf / inf, whose block alone has no scale.
    for row, col in ((900, 1031), (1999, 0)):
        block = col // 128
        assert bool(q[row, col].isnan()) and bool(s[row, block].isnan())
        others = torch.arange(1032) // 128 != block
        assert bool((q[row, others] == 0).all())
        assert bool((s[row, torch.arange(9) != block] == OO.TINY_SCALE).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(9000, 1032), (20000, 264), (1500, 8192)], ids=str)
def test_gradients_of_many_rows_a_block(shape, dtype):
    f64 = lambda t: t.double().cpu().numpy()
    h, dy, dh = (draw(shape, dtype, s) for s in (20, 21, 22))
    w = draw((shape[1],), "f32", 23)
    dx, dw = T.rmsnorm_grad(dy, h, w, dh=dh, workspace=T.rmsnorm_grad_workspace(h))
    rx, rw, bx, bw = OO.rmsnorm_grad(f64(dy), f64(h), f64(w), f64(dh))
    for got, ref, bound, kind, rel in ((dx, rx, bx, dtype, 2.0 ** -18), (dw, rw, bw, "f32", 2.0 ** -14)):
        ok, worst, idx = OT.check(f64(got), ref, bound, kind, rel)
        assert ok, (worst, idx)
