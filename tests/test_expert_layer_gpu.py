"""The expert-layer example against the float64 definitions, end to end."""

import numpy as np
import pytest

from oracle import operators as OO

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402
from examples.expert_layer import ExpertLayer, main  # noqa: E402


def f64(t):
    return t.double().cpu().numpy()


def relative(got, want):
    return np.linalg.norm(f64(got) - want) / np.linalg.norm(want)


def inputs(rows, hidden, width):
    g = torch.Generator(device="cuda").manual_seed(5)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    return normal(rows, hidden), normal(rows, hidden), normal(rows, width), normal(rows, hidden)


@pytest.mark.parametrize("rows", [1, 40, 700])
def test_serving_step(rows):
    layer = ExpertLayer(512, 384, 5)
    x, r, _, _ = inputs(rows, 512, 384)
    y, h = layer.serve(x, r)
    T.check(layer.workspace)
    order, offsets = layer.route(h)
    order, off = order.cpu().numpy(), offsets.tolist()
    # The same 8-bit rows and weights, multiplied in 64 bits.
    q, s, _ = T.rmsnorm_fp8(x, layer.norm, residual=r)
    want, _ = OO.gemm_fp8(f64(q), f64(s), *(f64(t) for t in layer.shared8))
    e, _ = OO.grouped_fp8(f64(q)[order], f64(s)[order], *(f64(t) for t in layer.weights8), off)
    want[order] += e
    # Three roundings to bf16 (2^-9 each at most) of terms of similar size.
    assert relative(y, want) < 3 * 2.0 ** -9
    # And against the unquantised layer: e4m3 keeps 2^-4 of each factor.
    y64, _ = OO.rmsnorm(f64(x), f64(layer.norm), f64(r))
    full = np.zeros_like(want)
    full[order] = OO.grouped(y64[order], f64(layer.weights), off)[0]
    shared = f64(layer.shared8[0]) * OO.spread(OO.spread(f64(layer.shared8[1]), 384, 0), 512, 1)
    assert relative(y, full + y64 @ shared.T) < 2 * 2.0 ** -4


@pytest.mark.parametrize("rows", [3, 700])
def test_training_step(rows):
    layer = ExpertLayer(256, 320, 6)
    x, r, dout, dh = inputs(rows, 256, 320)
    out, dx, dnorm, dweights = layer.train_step(x, r, dout, dh)
    T.check(layer.workspace)
    y, h = T.rmsnorm(x, layer.norm, residual=r)
    order, offsets = layer.route(h)
    order, off = order.cpu().numpy(), offsets.tolist()
    want = np.zeros((rows, 320))
    want[order] = OO.grouped(f64(y)[order], f64(layer.weights), off)[0]
    assert relative(out, want) < 2.0 ** -8
    dw, _ = OO.wgrad(f64(y)[order], f64(dout)[order], off)
    assert relative(dweights, dw) < 2.0 ** -8
    dy = np.zeros((rows, 256))
    dy[order] = OO.grouped(f64(dout)[order], f64(layer.weights), off, trans_b=True)[0]
    rx, rn, _, _ = OO.rmsnorm_grad(dy, f64(h), f64(layer.norm), f64(dh))
    assert relative(dx, rx) < 2.0 ** -7          # dy and dx are each rounded to bf16
    assert relative(dnorm, rn) < 2.0 ** -8       # dy's rounding


def test_the_example_runs(capsys):
    assert main(["--rows", "64", "--hidden", "256", "--width", "128", "--experts", "4",
                 "--steps", "2"]) == 0
    assert "serve" in capsys.readouterr().out
