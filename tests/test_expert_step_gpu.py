"""A run of the routing, layer-norm and clipping operators together, as an expert
layer uses them, against the float64 definitions; and the example with several
experts a row."""

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


def normal(seed, *shape, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("tokens,k,padding", [(1, 2, 0), (37, 3, 5), (700, 2, 90)])
def test_a_training_step_of_an_expert_layer(tokens, k, padding):
    hidden, width, experts = 256, 136, 7
    x, r, dout, dh = (normal(i, tokens, n) for i, n in enumerate((hidden, hidden, width, hidden)))
    gamma, beta = 1 + normal(5, hidden, scale=0.1), normal(6, hidden, scale=0.1)
    w = normal(7, experts, hidden, width, scale=hidden ** -0.5)
    ids = torch.randint(0, experts, (tokens, k), generator=torch.Generator().manual_seed(8)).cuda()
    if padding:
        ids[-padding:] = -1
    p = normal(9, tokens, k, dtype=torch.float32).softmax(1)
    ws = T.workspace()

    y, h = T.layernorm(x, gamma, beta, residual=r)
    slots, offsets, order = T.expert_sort(ids, experts)
    # Rows of nobody hold NaNs: nothing may read them.
    rows = T.expert_dispatch(y, slots, out=torch.full((tokens * k, hidden), float("nan"),
                                                      dtype=y.dtype, device="cuda"))
    e = T.grouped_gemm(rows, w, offsets, workspace=ws,
                       out=torch.full((tokens * k, width), float("nan"), dtype=y.dtype, device="cuda"))
    out = T.expert_combine(e, slots, p)
    de, dp = T.expert_combine_grad(dout, e, slots, p)
    dw = T.grouped_wgrad(rows, de, offsets, out_dtype="f32", workspace=ws)
    drows = T.grouped_gemm(de, w, offsets, trans_b=True, workspace=ws)
    dy = T.expert_combine(drows, slots)
    dx, dgamma, dbeta = T.layernorm_grad(dy, h, gamma, dh=dh)
    grads = [dw, dgamma, dbeta]
    before = [f64(g) for g in grads]
    norm = T.clip_grads(grads, 0.5)
    T.check(ws)

    # Each step in 64 bits from what the step before left.
    sl, off = slots.cpu().numpy(), offsets.tolist()
    s64, o64, r64 = OO.expert_sort(ids.cpu().numpy(), experts)
    assert np.array_equal(sl, s64) and off == o64.tolist()
    assert np.array_equal(order.cpu().numpy(), r64)
    n = off[-1]
    assert n == (tokens - padding) * k
    y64, h64 = OO.layernorm(f64(x), f64(gamma), f64(beta), f64(r))
    assert relative(y, y64) < 2.0 ** -8 and relative(h, h64) < 2.0 ** -8
    assert np.array_equal(f64(rows)[:n], f64(y)[r64[:n] // k])
    e64 = OO.grouped(f64(rows), f64(w), off)[0]
    assert relative(e[:n], e64[:n]) < 2.0 ** -8 and bool(e[n:].isnan().all())
    assert relative(out, OO.expert_combine(f64(e), sl, f64(p))[0]) < 2.0 ** -8
    de64, dp64, mag = OO.expert_combine_grad(f64(dout), f64(e), sl, f64(p))
    assert relative(de[:n], de64[:n]) < 2.0 ** -8
    assert np.all(np.abs(f64(dp) - dp64) <= 2.0 ** -18 * mag)
    assert relative(dw * 1.0, OO.wgrad(f64(rows), f64(de), off)[0] * min(1, 0.5 / (float(norm) + 1e-6))) < 2.0 ** -17
    dr64 = OO.grouped(f64(de), f64(w), off, trans_b=True)[0]
    assert relative(drows[:n], dr64[:n]) < 2.0 ** -8
    assert relative(dy, OO.expert_combine(f64(drows), sl)[0]) < 2.0 ** -8
    if padding:
        assert not out[-padding:].any() and not dy[-padding:].any() and not dp[-padding:].any()
    dx64, dg64, db64 = OO.layernorm_grad(f64(dy), f64(h), f64(gamma), f64(dh))
    assert relative(dx, dx64) < 2.0 ** -8
    assert np.linalg.norm(before[1] - dg64) <= 2.0 ** -17 * np.linalg.norm(dg64) + 1e-12
    want, clipped = OO.clip(before, 0.5)
    assert abs(float(norm) - want) <= 2.0 ** -18 * want
    for g, c in zip(grads, clipped):
        assert np.linalg.norm(f64(g) - c) <= 2.0 ** -18 * np.linalg.norm(c)


def test_the_chain_s_gradients_against_differences():
    # loss = sum(combine(experts(dispatch(x))) * dout) in 64 bits, its differences in x
    # and in the weights against the operators' gradients in fp32 (the products,
    # which have no fp32 form, in 64 bits on the host).
    rng = np.random.default_rng(2)
    tokens, k, hidden, width, experts = 6, 2, 12, 20, 4
    ids = rng.integers(-1, experts, (tokens, k))
    x, w = rng.normal(size=(tokens, hidden)), rng.normal(size=(experts, hidden, width))
    p, dout = rng.random((tokens, k)), rng.normal(size=(tokens, width))
    slots, offsets, _ = OO.expert_sort(ids, experts)
    off = offsets.tolist()

    def loss(x, p):
        rows = OO.expert_dispatch(x, slots, tokens * k, fill=0.0)
        return (OO.expert_combine(OO.grouped(rows, w, off)[0], slots, p)[0] * dout).sum()

    def gpu(a):
        return torch.tensor(a, dtype=torch.float32, device="cuda")

    got, _, _ = T.expert_sort(torch.tensor(ids, device="cuda"), experts)
    assert np.array_equal(got.cpu().numpy(), slots)
    rows = T.expert_dispatch(gpu(x), got, out=torch.zeros(tokens * k, hidden, device="cuda"))
    e = OO.grouped(f64(rows), w, off)[0]
    de, dp = T.expert_combine_grad(gpu(dout), gpu(e), got, gpu(p),
                                   drows_out=torch.zeros(tokens * k, width, device="cuda"))
    drows = OO.grouped(f64(de), w, off, trans_b=True)[0]
    dx = T.expert_combine(gpu(drows), got)
    step = 1e-5
    for grad, at, other in ((dx, x, lambda v: loss(v, p)), (dp, p, lambda v: loss(x, v))):
        for i in np.ndindex(at.shape):
            up, down = at.copy(), at.copy()
            up[i] += step
            down[i] -= step
            # fp32 operands: 2^-24 of sums of a few dozen terms of size ten.
            assert abs((other(up) - other(down)) / (2 * step) - float(grad[i])) < 2e-4


@pytest.mark.parametrize("rows", [1, 40, 700])
def test_the_example_with_two_experts_a_row(rows):
    layer = ExpertLayer(512, 384, 5, choices=2)
    x, r, dout, dh = (normal(20 + i, rows, n) for i, n in enumerate((512, 512, 384, 512)))
    y, h = layer.serve(x, r)
    T.check(layer.workspace)
    experts, p = layer.choose(h)
    slots, off, _ = OO.expert_sort(experts.cpu().numpy(), 5)
    q, s, _ = T.rmsnorm_fp8(x, layer.norm, residual=r)
    want, _ = OO.gemm_fp8(f64(q), f64(s), *(f64(t) for t in layer.shared8))
    e, _ = OO.grouped_fp8(OO.expert_dispatch(f64(q), slots, 2 * rows),
                          OO.expert_dispatch(f64(s), slots, 2 * rows),
                          *(f64(t) for t in layer.weights8), off.tolist())
    want = want + OO.expert_combine(e, slots, f64(p))[0]
    # Four roundings to bf16 (2^-9 each at most) of terms of similar size.
    assert relative(y, want) < 4 * 2.0 ** -9

    out, dx, dnorm, dweights, drouter = layer.train_step(x, r, dout, dh)
    T.check(layer.workspace)
    yn, h = T.rmsnorm(x, layer.norm, residual=r)
    experts, p = layer.choose(h)
    slots, off, _ = OO.expert_sort(experts.cpu().numpy(), 5)
    off, p64, w64 = off.tolist(), f64(p), f64(layer.weights)
    rows64 = OO.expert_dispatch(f64(yn), slots, 2 * rows)
    e64 = OO.grouped(rows64, w64, off)[0]
    assert relative(out, OO.expert_combine(e64, slots, p64)[0]) < 2 * 2.0 ** -8
    de, dp, _ = OO.expert_combine_grad(f64(dout), e64, slots, p64)
    assert relative(dweights, OO.wgrad(rows64, de, off)[0]) < 2 * 2.0 ** -8
    dy = OO.expert_combine(OO.grouped(de, w64, off, trans_b=True)[0], slots)[0]
    dl = np.zeros((rows, 5))
    np.put_along_axis(dl, experts.cpu().numpy(), p64 * (dp - (p64 * dp).sum(1, keepdims=True)), 1)
    # The chosen logits' gradients cancel against their mean: relative to what cancels.
    size = np.linalg.norm(np.abs(f64(h)).T @ (np.abs(p64 * dp).sum(1, keepdims=True) * np.ones((1, 5))))
    assert np.linalg.norm(f64(drouter) - f64(h).T @ dl) < 2.0 ** -8 * size
    dx64, dn64, _, _ = OO.rmsnorm_grad(dy, f64(h), f64(layer.norm), f64(dh) + dl @ f64(layer.router).T)
    assert relative(dx, dx64) < 2.0 ** -6        # e, de, drows, dy, dh and dx are each rounded to bf16
    assert relative(dnorm, dn64) < 2.0 ** -6


def test_the_example_runs_with_two_experts_a_row(capsys):
    assert main(["--rows", "64", "--hidden", "256", "--width", "128", "--experts", "4",
                 "--choices", "2", "--steps", "2"]) == 0
    assert "train step" in capsys.readouterr().out
