"""Host-side checks of the layer norm, routing and clipping operators (no GPU):
the float64 definitions against differences and against each other, the
refusals that come before any CUDA call, and those of the Python functions."""

import ctypes as C

import numpy as np
import pytest

from oracle import operators as OO
from tile_size_decision_gb300 import _abi

torch = pytest.importorskip("torch")

import tile_size_decision_gb300 as T  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    from tile_size_decision_gb300 import build
    build.build()
    return _abi.load()


# ---- the definitions -------------------------------------------------------------------


def test_layernorm_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, r = rng.normal(size=(3, 11)), rng.normal(size=(3, 11))
    w, b = rng.normal(size=11), rng.normal(size=11)
    dy, dh = rng.normal(size=(3, 11)), rng.normal(size=(3, 11))

    def loss(x, w, b):
        y, h = OO.layernorm(x, w, b, r, eps=1e-3)
        return (y * dy).sum() + (h * dh).sum()

    grads = OO.layernorm_grad(dy, x + r, w, dh, eps=1e-3)
    step = 1e-5
    for which, (at, grad) in enumerate(zip((x, w, b), grads)):
        for i in np.ndindex(at.shape):
            up, down = [x, w, b], [x, w, b]
            up[which], down[which] = at.copy(), at.copy()
            up[which][i] += step
            down[which][i] -= step
            # Central differences: error O(step^2) plus rounding 1e-16 / step.
            assert abs((loss(*up) - loss(*down)) / (2 * step) - grad[i]) < 1e-8


def test_combine_gradients_against_differences():
    rng = np.random.default_rng(1)
    experts = np.array([[0, 2], [1, -1], [2, 0], [7, 1]])
    slots, offsets, order = OO.expert_sort(experts, 3)
    rows, w, dy = rng.normal(size=(8, 5)), rng.normal(size=(4, 2)), rng.normal(size=(4, 5))
    drows, dw, _ = OO.expert_combine_grad(dy, rows, slots, w, fill=0.0)
    # The sum is linear in each operand: a difference is exact to rounding.
    for i in np.ndindex(rows.shape):
        d = np.zeros_like(rows)
        d[i] = 1.0
        assert abs((OO.expert_combine(d, slots, w)[0] * dy).sum() - drows[i]) < 1e-12
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = 1.0
        assert abs((OO.expert_combine(rows, slots, d)[0] * dy).sum() - dw[i]) < 1e-12
    # And dispatch's gradient is the sum without weights.
    x = rng.normal(size=(4, 5))
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = 1.0
        got = (OO.expert_dispatch(d, slots, 8, fill=0.0) * rows).sum()
        assert abs(got - OO.expert_combine(rows, slots)[0][i]) < 1e-12


def test_sort_definition():
    experts = np.array([[2, 0], [0, 5], [-1, 2]])
    slots, offsets, order = OO.expert_sort(experts, 3)
    assert slots.tolist() == [[2, 0], [1, -1], [-1, 3]]
    assert offsets.tolist() == [0, 2, 2, 4]
    assert order.tolist() == [1, 2, 0, 5, -1, -1]


def test_clip_definition():
    norm, out = OO.clip([np.array([3.0]), np.array([4.0])], 1.0, eps=0.0)
    assert norm == 5.0 and np.allclose([o[0] for o in out], [0.6, 0.8])
    assert OO.clip([np.zeros(3)], 0.0, 0.0)[1][0].tolist() == [0, 0, 0]


# ---- refusals of the C calls ---------------------------------------------------------------

PTR = 0x10000


def fill(desc, kw, **more):
    for k, v in {**kw, **more}.items():
        setattr(desc, k, v)
    return desc


NORM = dict(rows=4, cols=64, x=PTR, weight=PTR, bias=PTR, y=PTR, ldx=64, ldy=64, eps=1e-5,
            dtype=_abi.BF16, weight_dtype=_abi.BF16, out_dtype=_abi.BF16)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), _abi.ERR_INVALID_ARG),
    (dict(cols=0), _abi.ERR_INVALID_ARG),
    (dict(rows=1 << 31), _abi.ERR_TOO_LARGE),
    (dict(x=None), _abi.ERR_INVALID_ARG),
    (dict(x=PTR + 1), _abi.ERR_MISALIGNED),
    (dict(weight=None), _abi.ERR_INVALID_ARG),
    (dict(bias=PTR + 1), _abi.ERR_MISALIGNED),
    (dict(weight_dtype=_abi.E4M3), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(dtype=9), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(out_dtype=_abi.F32), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(out_dtype=_abi.E4M3), _abi.ERR_INVALID_ARG),          # no scales
    (dict(ldx=63), _abi.ERR_INVALID_ARG),
    (dict(residual=PTR, ldr=10), _abi.ERR_INVALID_ARG),
    (dict(h=PTR + 1, ldh=64), _abi.ERR_MISALIGNED),
    (dict(y=None), _abi.ERR_INVALID_ARG),
])
def test_layernorm_refusals(lib, kw, status):
    d = fill(_abi.LayernormDesc(), NORM, **kw)
    assert lib.tiles_layernorm(C.byref(d), None) == status
    assert lib.tiles_last_error() != b""


@pytest.mark.parametrize("kw,status", [
    (dict(cols=0), _abi.ERR_INVALID_ARG),
    (dict(cols=(1 << 28) + 1), _abi.ERR_TOO_LARGE),
    (dict(dtype=_abi.E4M3), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(dweight=None), _abi.ERR_INVALID_ARG),
    (dict(dbias=None), _abi.ERR_INVALID_ARG),
    (dict(dbias=PTR + 2), _abi.ERR_INVALID_ARG),
    (dict(dy=None), _abi.ERR_INVALID_ARG),
    (dict(h=PTR + 1), _abi.ERR_MISALIGNED),
    (dict(lddx=5), _abi.ERR_INVALID_ARG),
    (dict(dh=PTR, lddh=5), _abi.ERR_INVALID_ARG),
    (dict(), _abi.ERR_INVALID_ARG),                             # no workspace
])
def test_layernorm_gradient_refusals(lib, kw, status):
    base = dict(rows=4, cols=64, dy=PTR, h=PTR, weight=PTR, dx=PTR, dweight=PTR, dbias=PTR, lddy=64,
                ldh=64, lddx=64, eps=1e-5, dtype=_abi.F16, weight_dtype=_abi.F32)
    d = fill(_abi.LayernormGradDesc(), base, **kw)
    assert lib.tiles_layernorm_grad(C.byref(d), None, 0, None) == status


SORT = dict(tokens=8, k=2, groups=4, experts=PTR, ld=2, slots=PTR, offsets=PTR, order=PTR,
            index_bytes=8)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), _abi.ERR_INVALID_ARG),
    (dict(k=0), _abi.ERR_INVALID_ARG),
    (dict(groups=0), _abi.ERR_INVALID_ARG),
    (dict(groups=4097), _abi.ERR_TOO_LARGE),
    (dict(tokens=(1 << 23) + 1), _abi.ERR_TOO_LARGE),
    (dict(tokens=1 << 62, k=4, ld=4), _abi.ERR_TOO_LARGE),
    (dict(index_bytes=2), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(experts=None), _abi.ERR_INVALID_ARG),
    (dict(experts=PTR + 4), _abi.ERR_MISALIGNED),
    (dict(slots=None), _abi.ERR_INVALID_ARG),
    (dict(offsets=None), _abi.ERR_INVALID_ARG),
    (dict(offsets=PTR + 2), _abi.ERR_INVALID_ARG),
    (dict(order=PTR + 1), _abi.ERR_MISALIGNED),
    (dict(ld=1), _abi.ERR_INVALID_ARG),
    (dict(tokens=10000), _abi.ERR_INVALID_ARG),                 # no workspace
])
def test_sort_refusals(lib, kw, status):
    d = fill(_abi.ExpertSortDesc(), SORT, **kw)
    assert lib.tiles_expert_sort(C.byref(d), None, 0, None) == status


def test_sort_workspaces(lib):
    size = lib.tiles_expert_sort_workspace_bytes
    assert size(0, 1, 1) >= 256 and size(16384, 8, 64) > 256
    for bad in ((-1, 2, 4), (4, 0, 4), (4, 2, 0), (4, 2, 4097), (1 << 24, 2, 4), (1 << 62, 4, 4)):
        assert size(*bad) == 0
    # A workspace that is too small, or starts off 16 bytes, is refused.
    d = fill(_abi.ExpertSortDesc(), SORT, tokens=16384, k=8, ld=8)
    need = size(16384, 8, 4)
    assert lib.tiles_expert_sort(C.byref(d), PTR, need - 1, None) == _abi.ERR_INVALID_ARG
    assert lib.tiles_expert_sort(C.byref(d), PTR + 4, need, None) == _abi.ERR_MISALIGNED


DISPATCH = dict(tokens=4, k=2, rows=8, cols=64, slots=PTR, x=PTR, out=PTR, ld_slots=2, ldx=64,
                ld_out=64, dtype=_abi.BF16)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), _abi.ERR_INVALID_ARG),
    (dict(k=0), _abi.ERR_INVALID_ARG),
    (dict(tokens=1 << 29, k=4, ld_slots=4), _abi.ERR_TOO_LARGE),
    (dict(rows=-1), _abi.ERR_INVALID_ARG),
    (dict(cols=0), _abi.ERR_INVALID_ARG),
    (dict(cols=1 << 31), _abi.ERR_TOO_LARGE),
    (dict(dtype=9), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(slots=None), _abi.ERR_INVALID_ARG),
    (dict(slots=PTR + 2), _abi.ERR_INVALID_ARG),
    (dict(ld_slots=1), _abi.ERR_INVALID_ARG),
    (dict(x=None), _abi.ERR_INVALID_ARG),
    (dict(out=PTR + 1), _abi.ERR_MISALIGNED),
    (dict(ld_out=60), _abi.ERR_INVALID_ARG),
    (dict(scales=PTR), _abi.ERR_INVALID_ARG),
    (dict(out_scales=PTR), _abi.ERR_INVALID_ARG),
    (dict(scales=PTR + 1, out_scales=PTR), _abi.ERR_MISALIGNED),
])
def test_dispatch_refusals(lib, kw, status):
    d = fill(_abi.DispatchDesc(), DISPATCH, **kw)
    assert lib.tiles_expert_dispatch(C.byref(d), None) == status


COMBINE = dict(tokens=4, k=2, rows=8, cols=64, slots=PTR, weights=PTR, in_=PTR, dy=PTR, out=PTR,
               dweights=PTR, ld_slots=2, ld_weights=2, ld_in=64, ld_dy=64, ld_out=64, ld_dweights=2,
               dtype=_abi.BF16, weight_dtype=_abi.F32)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), _abi.ERR_INVALID_ARG),
    (dict(cols=0), _abi.ERR_INVALID_ARG),
    (dict(dtype=_abi.E4M3), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(weight_dtype=_abi.E4M3), _abi.ERR_UNSUPPORTED_DTYPE),
    (dict(slots=None), _abi.ERR_INVALID_ARG),
    (dict(in_=None), _abi.ERR_INVALID_ARG),
    (dict(in_=PTR + 1), _abi.ERR_MISALIGNED),
    (dict(out=None), _abi.ERR_INVALID_ARG),
    (dict(ld_out=9), _abi.ERR_INVALID_ARG),
    (dict(weights=PTR + 2), _abi.ERR_MISALIGNED),
    (dict(ld_weights=1), _abi.ERR_INVALID_ARG),
])
def test_combine_refusals(lib, kw, status):
    d = fill(_abi.CombineDesc(), COMBINE, **kw)
    assert lib.tiles_expert_combine(C.byref(d), None) == status
    assert lib.tiles_expert_combine_grad(C.byref(d), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(weights=None), _abi.ERR_INVALID_ARG),
    (dict(dy=None), _abi.ERR_INVALID_ARG),
    (dict(ld_dy=9), _abi.ERR_INVALID_ARG),
    (dict(dweights=None), _abi.ERR_INVALID_ARG),
    (dict(dweights=PTR + 2), _abi.ERR_INVALID_ARG),
    (dict(ld_dweights=1), _abi.ERR_INVALID_ARG),
])
def test_combine_gradient_refusals(lib, kw, status):
    d = fill(_abi.CombineDesc(), COMBINE, **kw)
    assert lib.tiles_expert_combine_grad(C.byref(d), None) == status


def tensors(*specs):
    a = (_abi.GradTensor * len(specs))()
    for t, (grad, out, count, dtype) in zip(a, specs):
        t.grad, t.out, t.count, t.dtype = grad, out, count, dtype
    return a


@pytest.mark.parametrize("specs,max_norm,eps,status", [
    ([(PTR, None, 4, _abi.F32)], -1.0, 0.0, _abi.ERR_INVALID_ARG),
    ([(PTR, None, 4, _abi.F32)], float("nan"), 0.0, _abi.ERR_INVALID_ARG),
    ([(PTR, None, 4, _abi.F32)], 1.0, -1.0, _abi.ERR_INVALID_ARG),
    ([(PTR, None, 4, _abi.E4M3)], 1.0, 0.0, _abi.ERR_UNSUPPORTED_DTYPE),
    ([(PTR, None, -4, _abi.F32)], 1.0, 0.0, _abi.ERR_INVALID_ARG),
    ([(None, None, 4, _abi.F32)], 1.0, 0.0, _abi.ERR_INVALID_ARG),
    ([(PTR + 2, None, 4, _abi.F32)], 1.0, 0.0, _abi.ERR_MISALIGNED),
    ([(PTR, PTR + 0x101, 4, _abi.BF16)], 1.0, 0.0, _abi.ERR_MISALIGNED),
    ([(PTR, None, 1 << 41, _abi.F32)], 1.0, 0.0, _abi.ERR_TOO_LARGE),
    ([(PTR, None, 1 << 40, _abi.F32)] * 17, 1.0, 0.0, _abi.ERR_TOO_LARGE),
    # The same tensor twice; one that starts inside another; an output over
    # another gradient, over its own a little shifted, and over another output.
    ([(PTR, None, 4, _abi.F32)] * 2, 1.0, 0.0, _abi.ERR_INVALID_ARG),
    ([(PTR, None, 8, _abi.F32), (PTR + 16, None, 8, _abi.F32)], 1.0, 0.0, _abi.ERR_INVALID_ARG),
    ([(PTR, PTR + 64, 4, _abi.F32), (PTR + 64, PTR + 128, 4, _abi.F32)], 1.0, 0.0,
     _abi.ERR_INVALID_ARG),
    ([(PTR, PTR + 8, 4, _abi.F32)], 1.0, 0.0, _abi.ERR_INVALID_ARG),
    ([(PTR, PTR + 64, 4, _abi.F32), (PTR + 32, PTR + 64, 4, _abi.F32)], 1.0, 0.0,
     _abi.ERR_INVALID_ARG),
    # A large gradient that holds a later output's place, past one that ends early.
    ([(PTR, PTR + 0x1000, 256, _abi.F32), (PTR + 0x2000, PTR + 512, 1, _abi.F32)], 1.0, 0.0,
     _abi.ERR_INVALID_ARG),
])
def test_clip_refusals(lib, specs, max_norm, eps, status):
    a = tensors(*specs)
    assert lib.tiles_clip_grads(a, len(specs), max_norm, eps, PTR, PTR, 1 << 30, None) == status


def test_norm_refusals(lib):
    a = tensors((PTR, None, 4, _abi.F32))
    assert lib.tiles_grad_norm(a, -1, PTR, None, 0, None) == _abi.ERR_INVALID_ARG
    assert lib.tiles_grad_norm(None, 1, PTR, None, 0, None) == _abi.ERR_INVALID_ARG
    assert lib.tiles_grad_norm(a, 1, None, None, 0, None) == _abi.ERR_INVALID_ARG
    assert lib.tiles_grad_norm(a, 1, PTR + 2, None, 0, None) == _abi.ERR_INVALID_ARG
    assert lib.tiles_grad_norm(a, 1 << 21, PTR, None, 0, None) == _abi.ERR_TOO_LARGE
    assert lib.tiles_grad_norm_workspace_bytes(-1) == 0


def test_no_tokens_touch_nothing(lib):
    assert lib.tiles_expert_dispatch(C.byref(fill(_abi.DispatchDesc(), DISPATCH, tokens=0, x=None)),
                                     None) == _abi.OK
    d = fill(_abi.CombineDesc(), COMBINE, tokens=0, in_=None, out=None)
    assert lib.tiles_expert_combine(C.byref(d), None) == _abi.OK
    assert lib.tiles_expert_combine_grad(C.byref(d), None) == _abi.OK
    d = fill(_abi.LayernormDesc(), NORM, rows=0, x=None, y=None, weight=None)
    assert lib.tiles_layernorm(C.byref(d), None) == _abi.OK


def test_null_descriptors(lib):
    for fn in (lib.tiles_layernorm, lib.tiles_expert_dispatch, lib.tiles_expert_combine,
               lib.tiles_expert_combine_grad):
        assert fn(None, None) == _abi.ERR_INVALID_ARG
    for fn in (lib.tiles_layernorm_grad, lib.tiles_expert_sort):
        assert fn(None, None, 0, None) == _abi.ERR_INVALID_ARG
    assert lib.tiles_layernorm_grad_workspace_bytes(4, 0) == 0


@pytest.mark.parametrize("packer,desc", [
    ("_LAYERNORM", _abi.LayernormDesc), ("_LAYERNORM_GRAD", _abi.LayernormGradDesc),
    ("_SORT", _abi.ExpertSortDesc), ("_DISPATCH", _abi.DispatchDesc),
    ("_COMBINE", _abi.CombineDesc), ("_GRAD_TENSOR", _abi.GradTensor)])
def test_packed_descriptors_are_the_structures(packer, desc):
    packer = getattr(T, packer)
    assert packer.size == C.sizeof(desc)
    values = [i + 1 for i in range(len(desc._fields_))]
    d = desc.from_buffer_copy(packer.pack(*values))
    assert [getattr(d, name) for name, _ in desc._fields_] == values


# ---- refusals of the Python functions ---------------------------------------------------------


class On:
    """What the checks look at of a CUDA tensor, on GPU `device`."""

    is_cuda = True

    def __init__(self, device, *shape, dtype=torch.bfloat16):
        self.t = torch.zeros(shape, dtype=dtype)
        self.device_index = device

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device_index

    @property
    def device(self):
        return torch.device("cpu")          # where new outputs would go


F32, I32, I64, E4M3 = torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn


def calls(at):
    """The calls, with the GPUs that their operands are on, and how many operands each has."""
    def m(i, *shape, dtype=torch.bfloat16):
        return On(at[i % len(at)], *shape, dtype=dtype)

    return {
        "layernorm": (6, lambda: T.layernorm(m(0, 4, 16), m(1, 16), m(2, 16), residual=m(3, 4, 16),
                                             out=m(4, 4, 16), h_out=m(5, 4, 16))),
        "layernorm_fp8": (5, lambda: T.layernorm_fp8(
            m(0, 4, 16), m(1, 16), m(2, 16), out=m(3, 4, 16, dtype=E4M3),
            scales=m(4, 4, 1, dtype=F32))),
        "layernorm_grad": (7, lambda: T.layernorm_grad(
            m(0, 4, 16), m(1, 4, 16), m(2, 16), dh=m(3, 4, 16), dx_out=m(4, 4, 16),
            dweight_out=m(5, 16, dtype=F32), dbias_out=m(6, 16, dtype=F32))),
        "expert_sort": (1, lambda: T.expert_sort(m(0, 4, 2, dtype=I64), 3)),
        "expert_dispatch": (5, lambda: T.expert_dispatch(
            m(0, 4, 16), m(1, 4, 2, dtype=I32), scales=m(2, 4, 1, dtype=F32), out=m(3, 8, 16),
            scales_out=m(4, 8, 1, dtype=F32))),
        "expert_combine": (4, lambda: T.expert_combine(
            m(0, 8, 16), m(1, 4, 2, dtype=I32), m(2, 4, 2, dtype=F32), out=m(3, 4, 16))),
        "expert_combine_grad": (6, lambda: T.expert_combine_grad(
            m(0, 4, 16), m(1, 8, 16), m(2, 4, 2, dtype=I32), m(3, 4, 2), drows_out=m(4, 8, 16),
            dweights_out=m(5, 4, 2, dtype=F32))),
        "grad_norm": (2, lambda: T.grad_norm([m(0, 4, 16), m(1, 3, dtype=F32)])),
        "clip_grads": (4, lambda: T.clip_grads([m(0, 4, 16), m(1, 3, dtype=F32)], 1.0,
                                               out=[m(2, 4, 16), m(3, 3, dtype=F32)])),
    }


@pytest.mark.parametrize("name", sorted(calls([0])))
def test_operands_of_another_gpu_are_refused(name, monkeypatch):
    class Library:
        """Stands in for the library: sizes are given, whatever launches was taken."""

        def __getattr__(self, name):
            def call(*args):
                if name.endswith("workspace_bytes"):
                    return 256
                raise AssertionError(f"{name} was called")
            return call

    monkeypatch.setattr(T, "_CALLS", T._NoCalls)
    monkeypatch.setattr(T, "load", Library)
    monkeypatch.setattr(T, "_raw_stream", lambda stream: 0)
    monkeypatch.setattr(T, "_scratch", lambda *a: (None, 0, 256))
    monkeypatch.setattr(T, "_DEVICES", 2, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    count, call = calls([0])[name]
    with pytest.raises(AssertionError, match="was called"):
        call()
    for other in range(count):
        with pytest.raises(ValueError, match="current device"):
            calls([1 if i == other else 0 for i in range(count)])[name][1]()


def g(*shape, dtype=torch.bfloat16):
    return On(0, *shape, dtype=dtype)


def sl(*shape):
    return On(0, *shape, dtype=I32)


@pytest.mark.parametrize("kind,call", [
    (ValueError, lambda: T.layernorm(torch.zeros(4, 16), torch.zeros(16))),
    (ValueError, lambda: T.layernorm(g(4, 16), g(15))),
    (ValueError, lambda: T.layernorm(g(4, 16), g(16), g(15))),
    (TypeError, lambda: T.layernorm(g(4, 16), g(16), g(16, dtype=F32))),
    (TypeError, lambda: T.layernorm(g(4, 16), g(16), residual=g(4, 16, dtype=F32))),
    (ValueError, lambda: T.layernorm(g(4, 16), g(16), out=g(4, 15))),
    (ValueError, lambda: T.layernorm(g(16), g(16))),
    (TypeError, lambda: T.layernorm(g(4, 16, dtype=torch.float64), g(16))),
    (ValueError, lambda: T.layernorm_fp8(g(4, 16), g(16), scales=g(4, 2, dtype=F32))),
    (ValueError, lambda: T.layernorm_grad(g(4, 16), g(4, 15), g(15))),
    (TypeError, lambda: T.layernorm_grad(g(4, 16), g(4, 16), g(16), dweight_out=g(16))),
    (TypeError, lambda: T.expert_sort(g(4, 2), 4)),
    (ValueError, lambda: T.expert_sort(sl(4), 4)),
    (ValueError, lambda: T.expert_sort(torch.zeros((4, 2), dtype=I32), 4)),
    (T.TilesError, lambda: T.expert_sort(sl(4, 2), 0)),
    (T.TilesError, lambda: T.expert_sort(sl(4, 2), 5000)),
    (T.TilesError, lambda: T.expert_sort(sl(4, 0), 4)),
    (ValueError, lambda: T.expert_dispatch(g(4, 16), sl(5, 2))),
    (TypeError, lambda: T.expert_dispatch(g(4, 16), On(0, 4, 2, dtype=I64))),
    (TypeError, lambda: T.expert_dispatch(g(4, 16), sl(4, 2), out=g(8, 16, dtype=F32))),
    (ValueError, lambda: T.expert_dispatch(g(4, 16), sl(4, 2), out=g(8, 15))),
    (ValueError, lambda: T.expert_dispatch(g(4, 16), sl(4, 2), scales=g(4, 2, dtype=F32))),
    (ValueError, lambda: T.expert_dispatch(g(4, 16), sl(4, 2), scales_out=g(8, 1, dtype=F32))),
    (TypeError, lambda: T.expert_combine(g(8, 16, dtype=E4M3), sl(4, 2))),
    (ValueError, lambda: T.expert_combine(g(8, 16), sl(4, 2), g(4, 3))),
    (TypeError, lambda: T.expert_combine(g(8, 16), sl(4, 2), On(0, 4, 2, dtype=I32))),
    (ValueError, lambda: T.expert_combine(g(8, 16), sl(4, 2), out=g(5, 16))),
    (ValueError, lambda: T.expert_combine_grad(g(4, 15), g(8, 16), sl(4, 2), g(4, 2))),
    (TypeError, lambda: T.expert_combine_grad(g(4, 16), g(8, 16), sl(4, 2), g(4, 2),
                                              dweights_out=g(4, 2))),
    (ValueError, lambda: T.grad_norm([])),
    (ValueError, lambda: T.grad_norm([torch.zeros(3)])),
    (TypeError, lambda: T.grad_norm([g(3, dtype=I32)])),
    (TypeError, lambda: T.grad_norm([g(3), None])),
    (ValueError, lambda: T.clip_grads([g(3)], 1.0, out=[])),
    (ValueError, lambda: T.clip_grads([g(3)], 1.0, out=[g(4)])),
    (ValueError, lambda: T.clip_grads([g(3)], 1.0, out=[g(3, dtype=F32)])),
    (TypeError, lambda: T.clip_grads([g(3)], 1.0, out=[None])),
    (TypeError, lambda: T.clip_grads([g(3)], None)),
    (T.TilesError, lambda: T.clip_grads([g(3)], -1.0, workspace=g(1 << 16))),
])
def test_what_the_functions_refuse(lib, kind, call, monkeypatch):
    monkeypatch.setattr(T, "_CALLS", T._NoCalls)
    monkeypatch.setattr(T, "_DEVICES", 1, raising=False)
    monkeypatch.setattr(T, "_raw_stream", lambda stream: 0)
    sizes = {"tiles_layernorm_grad_workspace_bytes", "tiles_grad_norm_workspace_bytes"}

    class Library:
        """The library, with the sizes that it would ask a GPU for."""

        def __getattr__(self, name):
            return (lambda *a: 1 << 12) if name in sizes else getattr(lib, name)

    monkeypatch.setattr(T, "load", Library)
    with pytest.raises(kind):
        call()


def test_elements_that_lie_together():
    base = torch.zeros(4, 6, 8)
    for t in (base, base.permute(2, 0, 1), base[1:3], base[:1, :, :], torch.zeros(()), base[0, 0]):
        assert T._dense(t) == torch.ops.aten.is_non_overlapping_and_dense(t) is True
    for t in (base[:, 1:3], base[..., ::2], base[0].expand(3, 6, 8), base[:, :, 0]):
        assert not T._dense(t)


def test_the_compiled_calls_are_bound():
    compiled = T._compiled()
    assert compiled is not T._NoCalls
    for name in ("layernorm", "layernorm_grad", "expert_sort", "expert_dispatch", "expert_combine",
                 "expert_combine_grad", "clip_grads"):
        assert getattr(T._NoCalls, name)() is None
        assert getattr(compiled, name)() is None
        assert getattr(compiled, name)(*[None] * 6) is None
