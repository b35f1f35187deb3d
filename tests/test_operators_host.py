"""Host-side checks of the norm, 8-bit and grouped operators (no GPU): the
float64 definitions against differences and against each other, and the
refusals that come before any CUDA call."""

import ctypes as C

import numpy as np
import pytest

from oracle import operators as OO
from tile_size_decision_gb300 import _abi


@pytest.fixture(scope="module")
def lib():
    from tile_size_decision_gb300 import build
    build.build()
    return _abi.load()


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, r = rng.normal(size=(3, 11)), rng.normal(size=(3, 11))
    w, dy, dh = rng.normal(size=11), rng.normal(size=(3, 11)), rng.normal(size=(3, 11))

    def loss(x, r, w):
        y, h = OO.rmsnorm(x, w, r, eps=1e-3)
        return (y * dy).sum() + (h * dh).sum()

    dx, dw, _, _ = OO.rmsnorm_grad(dy, x + r, w, dh, eps=1e-3)
    step = 1e-5
    for i in range(3):
        for j in range(11):
            d = np.zeros_like(x)
            d[i, j] = step
            # Central differences: error O(step^2) plus rounding 1e-16 / step.
            num = (loss(x + d, r, w) - loss(x - d, r, w)) / (2 * step)
            assert abs(num - dx[i, j]) < 1e-8
            num = (loss(x, r + d, w) - loss(x, r - d, w)) / (2 * step)
            assert abs(num - dx[i, j]) < 1e-8
    for j in range(11):
        d = np.zeros_like(w)
        d[j] = step
        assert abs((loss(x, r, w + d) - loss(x, r, w - d)) / (2 * step) - dw[j]) < 1e-8


def test_grouped_gradients_against_differences():
    rng = np.random.default_rng(1)
    off = [0, 2, 2, 5]
    a, w, dc = rng.normal(size=(5, 3)), rng.normal(size=(3, 3, 4)), rng.normal(size=(5, 4))
    da, _ = OO.grouped(dc, w, off, trans_b=True)
    dw, _ = OO.wgrad(a, dc, off)
    # The product is linear in each operand: a difference is exact to rounding.
    for idx in np.ndindex(a.shape):
        d = np.zeros_like(a)
        d[idx] = 1.0
        assert abs((OO.grouped(d, w, off)[0] * dc).sum() - da[idx]) < 1e-12
    for idx in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[idx] = 1.0
        assert abs((OO.grouped(a, d, off)[0] * dc).sum() - dw[idx]) < 1e-12


def test_block_scales_of_short_and_zero_blocks():
    y = np.zeros((2, 130))
    y[0, 129] = -896.0
    s = OO.row_scales(y)
    assert s.shape == (2, 2) and s[0, 1] == 2.0 and s[0, 0] == OO.TINY_SCALE
    sq = OO.square_scales(y)
    assert sq.shape == (1, 2) and sq[0, 1] == 2.0
    # Spacing of e4m3: 2^-3 of the leading power, 2^-9 below 2^-6.
    assert OO.half_step(np.array([1.5]))[0] == 2.0 ** -4
    assert OO.half_step(np.array([448.0]))[0] == 16.0
    assert OO.half_step(np.array([0.0]))[0] == 2.0 ** -10


PTR = 0x10000


def fill(desc, kw, **more):
    for k, v in {**kw, **more}.items():
        setattr(desc, k, v)
    return desc


NORM = dict(rows=4, cols=64, x=PTR, weight=PTR, y=PTR, ldx=64, ldy=64, eps=1e-6, dtype=_abi.BF16,
            weight_dtype=_abi.BF16, out_dtype=_abi.BF16)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), _abi.ERR_INVALID_ARG),
    (dict(cols=0), _abi.ERR_INVALID_ARG),
    (dict(rows=1 << 31), _abi.ERR_TOO_LARGE),
    (dict(x=None), _abi.ERR_INVALID_ARG),
    (dict(x=PTR + 1), _abi.ERR_MISALIGNED),
    (dict(weight=None), _abi.ERR_INVALID_ARG),
    (dict(weight_dtype=_abi.E4M3), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(dtype=9), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(out_dtype=_abi.F32), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(out_dtype=_abi.E4M3), _abi.ERR_INVALID_ARG),          # no scales
    (dict(ldx=63), _abi.ERR_INVALID_ARG),
    (dict(residual=PTR, ldr=10), _abi.ERR_INVALID_ARG),
    (dict(h=PTR + 1, ldh=64), _abi.ERR_MISALIGNED),
    (dict(y=None), _abi.ERR_INVALID_ARG),
])
def test_norm_refusals(lib, kw, status):
    d = fill(_abi.RmsnormDesc(), NORM, **kw)
    assert lib.tiles_rmsnorm(C.byref(d), None) == status
    assert lib.tiles_last_error() != b""


def test_norm_of_no_rows_touches_nothing(lib):
    d = fill(_abi.RmsnormDesc(), NORM, rows=0, x=None, y=None, weight=None)
    assert lib.tiles_rmsnorm(C.byref(d), None) == _abi.OK


@pytest.mark.parametrize("kw,status", [
    (dict(cols=0), _abi.ERR_INVALID_ARG),
    (dict(dtype=_abi.E4M3), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(dweight=None), _abi.ERR_INVALID_ARG),
    (dict(dy=None), _abi.ERR_INVALID_ARG),
    (dict(h=PTR + 1), _abi.ERR_MISALIGNED),
    (dict(lddx=5), _abi.ERR_INVALID_ARG),
    (dict(dh=PTR, lddh=5), _abi.ERR_INVALID_ARG),
    (dict(), _abi.ERR_INVALID_ARG),                             # no workspace
])
def test_norm_gradient_refusals(lib, kw, status):
    base = dict(rows=4, cols=64, dy=PTR, h=PTR, weight=PTR, dx=PTR, dweight=PTR, lddy=64, ldh=64,
                lddx=64, eps=1e-6, dtype=_abi.F16, weight_dtype=_abi.F32)
    d = fill(_abi.RmsnormGradDesc(), base, **kw)
    assert lib.tiles_rmsnorm_grad(C.byref(d), None, 0, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(block_rows=64), _abi.ERR_INVALID_ARG),
    (dict(dtype=_abi.E4M3), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(x=None), _abi.ERR_INVALID_ARG),
    (dict(ldq=60), _abi.ERR_INVALID_ARG),
    (dict(scales=None), _abi.ERR_INVALID_ARG),
    (dict(batch=-1), _abi.ERR_INVALID_ARG),
])
def test_quantise_refusals(lib, kw, status):
    base = dict(batch=1, rows=4, cols=64, x=PTR, q=PTR, scales=PTR, ldx=64, ldq=64, scale_row=1,
                scale_col=4, dtype=_abi.F16, block_rows=1)
    d = fill(_abi.QuantizeDesc(), base, **kw)
    assert lib.tiles_quantize_fp8(C.byref(d), None) == status


FP8 = dict(m=4, n=64, k=64, a=PTR, b=PTR, c=PTR, a_scales=PTR, b_scales=PTR, lda=64, ldb=64,
           ldc=64, in_dtype=_abi.E4M3, out_dtype=_abi.BF16, b_layout=_abi.B_NK)
GROUPED = dict(m=4, n=64, k=64, groups=2, offsets=PTR, a=PTR, b=PTR, c=PTR, lda=64, ldb=64, ldc=64,
               stride_b=4096, in_dtype=_abi.BF16, out_dtype=_abi.BF16, b_layout=_abi.B_KN)


@pytest.mark.parametrize("kw,status", [
    (dict(k=0), _abi.ERR_INVALID_ARG),
    (dict(m=-1), _abi.ERR_INVALID_ARG),
    (dict(n=1 << 31), _abi.ERR_TOO_LARGE),
    (dict(in_dtype=_abi.BF16), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(out_dtype=_abi.E4M3), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(b_layout=_abi.B_KN), _abi.ERR_INVALID_ARG),
    (dict(b_layout=5), _abi.ERR_INVALID_ARG),
    (dict(groups=1), _abi.ERR_INVALID_ARG),
    (dict(a_scales=None), _abi.ERR_INVALID_ARG),
    (dict(a=PTR + 8), _abi.ERR_MISALIGNED),
    (dict(lda=72), _abi.ERR_MISALIGNED),
    (dict(ldb=32), _abi.ERR_INVALID_ARG),
    (dict(c=PTR + 1), _abi.ERR_MISALIGNED),
    (dict(b_scales=PTR + 2), _abi.ERR_MISALIGNED),
    (dict(), _abi.ERR_INVALID_ARG),                             # no workspace
])
def test_dense_8bit_refusals(lib, kw, status):
    d = fill(_abi.ProductDesc(), FP8, **kw)
    assert lib.tiles_gemm_fp8(C.byref(d), None, 0, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(groups=0), _abi.ERR_INVALID_ARG),
    (dict(groups=5000), _abi.ERR_TOO_LARGE),
    (dict(offsets=None), _abi.ERR_INVALID_ARG),
    (dict(in_dtype=_abi.F32), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(stride_b=100), _abi.ERR_INVALID_ARG),
    (dict(stride_b=4100), _abi.ERR_MISALIGNED),
    (dict(lda=68), _abi.ERR_MISALIGNED),
    (dict(ldc=60), _abi.ERR_INVALID_ARG),
    (dict(), _abi.ERR_INVALID_ARG),                             # no workspace
])
def test_grouped_refusals(lib, kw, status):
    d = fill(_abi.ProductDesc(), GROUPED, **kw)
    assert lib.tiles_grouped_gemm(C.byref(d), None, 0, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(groups=0), _abi.ERR_INVALID_ARG),
    (dict(dw=None), _abi.ERR_INVALID_ARG),
    (dict(in_dtype=_abi.E4M3), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(out_dtype=_abi.E4M3), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(lddc=60), _abi.ERR_INVALID_ARG),
    (dict(lda=68), _abi.ERR_MISALIGNED),
    (dict(stride_dw=9), _abi.ERR_INVALID_ARG),
    (dict(), _abi.ERR_INVALID_ARG),                             # no workspace
])
def test_wgrad_refusals(lib, kw, status):
    base = dict(m=4, n=64, k=64, groups=2, offsets=PTR, a=PTR, dc=PTR, dw=PTR, lda=64, lddc=64,
                lddw=64, stride_dw=4096, in_dtype=_abi.F16, out_dtype=_abi.F32)
    d = fill(_abi.WgradDesc(), base, **kw)
    assert lib.tiles_grouped_wgrad(C.byref(d), None, 0, None) == status


def test_null_descriptors(lib):
    assert lib.tiles_rmsnorm(None, None) == _abi.ERR_INVALID_ARG
    assert lib.tiles_rmsnorm_grad(None, None, 0, None) == _abi.ERR_INVALID_ARG
    assert lib.tiles_quantize_fp8(None, None) == _abi.ERR_INVALID_ARG
    for fn in (lib.tiles_gemm_fp8, lib.tiles_grouped_gemm, lib.tiles_grouped_wgrad):
        assert fn(None, None, 0, None) == _abi.ERR_INVALID_ARG
    assert lib.tiles_rmsnorm_grad_workspace_bytes(4, 0) == 0


@pytest.mark.parametrize("packer,desc", [
    ("_NORM", _abi.RmsnormDesc), ("_NORM_GRAD", _abi.RmsnormGradDesc),
    ("_PRODUCT", _abi.ProductDesc), ("_WGRAD", _abi.WgradDesc)])
def test_packed_descriptors_are_the_structures(packer, desc):
    # The binding packs a descriptor's fields in order; every field must land
    # on its own in the structure the header declares.
    import tile_size_decision_gb300 as T
    packer = getattr(T, packer)
    assert packer.size == C.sizeof(desc)
    values = [i + 1 for i in range(len(desc._fields_))]
    d = desc.from_buffer_copy(packer.pack(*values))
    assert [getattr(d, name) for name, _ in desc._fields_] == values
