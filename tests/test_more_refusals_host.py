"""Operands of the layer norm, routing and clipping calls that are no tensors are refused by
name (no GPU: nothing is launched)."""

import pytest

torch = pytest.importorskip("torch")

import tile_size_decision_gb300 as T  # noqa: E402

F32, I32 = torch.float32, torch.int32


class OnGpu(torch.Tensor):
    """A tensor of the host that says it is on a GPU."""

    @property
    def is_cuda(self):
        return True


def m(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


X, W, SLOTS, ROWS, P = m(4, 16), m(16), m(4, 2, dtype=I32), m(8, 16), m(4, 2, dtype=F32)
NEEDED = [
    (T.layernorm, dict(x=X, weight=W)),
    (T.layernorm_fp8, dict(x=X, weight=W)),
    (T.layernorm_grad_workspace, dict(x=X)),
    (T.layernorm_grad, dict(dy=X, h=X, weight=W)),
    (T.expert_sort, dict(experts=SLOTS)),
    (T.expert_dispatch, dict(x=X, slots=SLOTS)),
    (T.expert_combine, dict(rows=ROWS, slots=SLOTS)),
    (T.expert_combine_grad, dict(dy=X, rows=ROWS, slots=SLOTS, weights=P)),
]
OTHERS = {T.layernorm: ("bias", "residual", "out", "h_out"),
          T.layernorm_fp8: ("bias", "residual", "out", "scales", "h_out"),
          T.layernorm_grad: ("dh", "dx_out", "dweight_out", "dbias_out"),
          T.expert_dispatch: ("scales", "out"),
          T.expert_combine: ("weights", "out"),
          T.expert_combine_grad: ("drows_out", "dweights_out")}


class Library:
    """Stands in for the library: nothing may come as far."""

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace_bytes"):
                return 256
            raise AssertionError(f"{name} was called")
        return call


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    monkeypatch.setattr(T, "_CALLS", T._NoCalls)
    monkeypatch.setattr(T, "load", Library)
    monkeypatch.setattr(T, "_raw_stream", lambda stream: 0)
    monkeypatch.setattr(T, "_DEVICES", 1, raising=False)


def call(fn, operands):
    return fn(**operands, **({"groups": 4} if fn is T.expert_sort else {}))


@pytest.mark.parametrize("value", [None, [[1.0]], 3, "x"], ids=str)
@pytest.mark.parametrize("fn,name", [(f, n) for f, ops in NEEDED for n in ops],
                         ids=lambda p: p if isinstance(p, str) else p.__name__)
def test_a_needed_operand_that_is_no_tensor(fn, name, value):
    operands = dict(next(ops for f, ops in NEEDED if f is fn))
    operands[name] = value
    with pytest.raises(TypeError, match=rf"^{name} must be a tensor"):
        call(fn, operands)


@pytest.mark.parametrize("value", [[[1.0]], 3, "x"], ids=str)
@pytest.mark.parametrize("fn,name", [(f, n) for f in OTHERS for n in OTHERS[f]],
                         ids=lambda p: p if isinstance(p, str) else p.__name__)
def test_another_operand_that_is_no_tensor(fn, name, value):
    operands = dict(next(ops for f, ops in NEEDED if f is fn))
    operands[name] = value
    with pytest.raises(TypeError, match=rf"^{name} must be a tensor"):
        call(fn, operands)


@pytest.mark.parametrize("value", [None, 3], ids=str)
def test_gradients_that_are_no_tensors(value):
    for run, name in ((lambda: T.grad_norm(value), "grads"), (lambda: T.clip_grads(value, 1.0), "grads"),
                      (lambda: T.grad_norm([X, value]), r"grads\[1\]"),
                      (lambda: T.clip_grads([X], 1.0, out=[value]), r"out\[0\]")):
        with pytest.raises(TypeError, match=rf"^{name} must be "):
            run()
    if value is not None:
        with pytest.raises(TypeError, match="^out must be "):
            T.clip_grads([X], 1.0, out=value)
