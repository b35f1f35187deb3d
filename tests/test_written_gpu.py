"""GPU tests of what autograd learns of the calls that write into tensors of the caller's:
their versions go up, as after any operation in place, so that a backward pass that would
need the old values says so."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402

F32 = torch.float32


@pytest.fixture(params=[True, False], ids=["compiled", "python"])
def way(request, monkeypatch):
    assert T._compiled() is not T._NoCalls
    if not request.param:
        monkeypatch.setattr(T, "_CALLS", T._NoCalls)


def draw(*shape, dtype=torch.bfloat16, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def calls():
    """By name: what a call reads, what it writes, and the call."""
    x, r, w, p = draw(6, 256), draw(6, 256, seed=2), draw(256, seed=3), draw(6, 2, dtype=F32, seed=4)
    rows, out, hh = draw(12, 256, seed=5), draw(6, 256), draw(6, 256)
    q, s = T.quantize_fp8(x)
    q8, s8 = torch.empty_like(q), torch.empty(6, 2, device="cuda")
    qr, sr = torch.zeros(12, 256, dtype=torch.uint8, device="cuda").view(q.dtype), torch.zeros(12, 2, device="cuda")
    dw, db, dp = (torch.empty(n, device="cuda") for n in (256, 256, (6, 2)))
    wide = draw(12, 256)
    slots = torch.arange(12, dtype=torch.int32, device="cuda").view(6, 2)
    g = [draw(500), draw(7, 9, dtype=F32), draw(0)]
    other = [torch.empty_like(t) for t in g]
    return {
        "norm": ([x, r, w], [out, hh], lambda: T.layernorm(x, w, residual=r, out=out, h_out=hh)),
        "norm in place": ([x, w], [r], lambda: T.layernorm(x, w, residual=r, h_out=r)),
        "norm alone": ([x, r, w], [], lambda: T.layernorm(x, w, residual=r)),
        "norm to 8 bits": ([x, w], [q8, s8, hh], lambda: T.layernorm_fp8(x, w, out=q8, scales=s8, h_out=hh)),
        "norm grad": ([x, r, w], [out, dw, db], lambda: T.layernorm_grad(
            x, r, w, dx_out=out, dweight_out=dw, dbias_out=db)),
        "dispatch": ([x, slots], [wide], lambda: T.expert_dispatch(x, slots, out=wide)),
        "dispatch of 8 bits": ([q, s, slots], [qr, sr], lambda: T.expert_dispatch(
            q, slots, scales=s, out=qr, scales_out=sr)),
        "combine": ([rows, slots, p], [out], lambda: T.expert_combine(rows, slots, p, out=out)),
        "combine grad": ([x, rows, slots, p], [wide, dp], lambda: T.expert_combine_grad(
            x, rows, slots, p, drows_out=wide, dweights_out=dp)),
        "grad norm": (g, [], lambda: T.grad_norm(g)),
        "clip": ([], g, lambda: T.clip_grads(g, 0.5)),
        "clip apart": (g, other, lambda: T.clip_grads(g, 0.5, out=other)),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_versions(name, way):
    read, written, call = calls()[name]
    was = [t._version for t in read], [t._version for t in written]
    call()
    assert [t._version for t in read] == was[0]
    assert all(t._version > v for t, v in zip(written, was[1]))
    # Tensors without a version are taken all the same.
    with torch.inference_mode():
        read, written, call = calls()[name]
        call()
    call()


@pytest.mark.parametrize("plain", [True, False])
def test_a_backward_pass_that_needs_the_values_before(plain, way):
    p = torch.nn.Parameter(draw(64, dtype=F32))
    grad, = torch.autograd.grad((p ** 3).sum(), p, create_graph=True)
    loss = (grad * grad).sum()                       # its gradient is made of grad's values
    if plain:
        with torch.no_grad():
            grad.mul_(0.5)
    else:
        T.clip_grads([grad], 0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_a_parameter_itself(way):
    p = torch.nn.Parameter(draw(3000, dtype=F32))
    before, v = p.detach().clone(), p._version
    norm = T.clip_grads([p], 1e-3)
    assert p.requires_grad and p.is_leaf and p.grad_fn is None and p._version > v
    # Two roundings of the factor and one of the product; the norm is within 34 * 2^-24.
    want = before.double() * (1e-3 / (before.double().norm() + 1e-6))
    assert bool(((p.detach().double() - want).abs() <= 38 * 2.0 ** -24 * want.abs()).all())
    assert abs(float(norm) - float(before.double().norm())) <= 34 * 2.0 ** -24 * float(norm)
