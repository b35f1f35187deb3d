"""GPU tests of calls whose operands are still being written when they are made: a busy
stream, every operand written in place there after that, and the call directly behind.
Each operand starts as other values that the call may take, so that a call on another
stream, or a kernel that reads before it has waited for what wrote its operands, gives
another result than the same call on operands that were there before.

They are written by PyTorch's copies and by a call of this library, whose kernel lets the
next one start before it has ended."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def draw(*shape, dtype=BF16, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def ids(tokens, k, groups, dtype=torch.int64, seed=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, groups, (tokens, k), generator=g, device="cuda").to(dtype)


def slots(tokens, k, seed=3):
    return T.expert_sort(ids(tokens, k, 7, seed=seed), 7)[0]


def norm(rows, cols, call=None, **more):
    ops = {"x": draw(rows, cols, seed=4), "weight": draw(cols, seed=5), "bias": draw(cols, seed=6),
           "residual": draw(rows, cols, seed=7)}
    return ops, lambda x, weight, bias, residual, **kw: (call or T.layernorm)(
        x, weight, bias, residual=residual, **kw)


def norm_grad(rows, cols, dtype=BF16):
    ops = {"dy": draw(rows, cols, dtype=dtype, seed=8), "h": draw(rows, cols, dtype=dtype, seed=9),
           "weight": draw(cols, dtype=dtype, seed=10), "dh": draw(rows, cols, dtype=dtype, seed=11)}
    return ops, lambda dy, h, weight, dh, **kw: T.layernorm_grad(dy, h, weight, dh=dh, **kw)


def sort(tokens, k, groups, dtype=torch.int64):
    return {"experts": ids(tokens, k, groups, dtype)}, \
        lambda experts, **kw: T.expert_sort(experts, groups, **kw)


def dispatch(tokens, k, cols):
    return {"x": draw(tokens, cols, seed=12), "slots": slots(tokens, k)}, T.expert_dispatch


def dispatch_fp8(tokens, k, cols):
    q, s = T.quantize_fp8(draw(tokens, cols, seed=13))
    return {"x": q.contiguous(), "slots": slots(tokens, k), "scales": s.contiguous()}, T.expert_dispatch


def combine(tokens, k, cols):
    return {"rows": draw(tokens * k, cols, seed=14), "slots": slots(tokens, k),
            "weights": draw(tokens, k, dtype=F32, seed=15)}, T.expert_combine


def combine_grad(tokens, k, cols):
    ops, _ = combine(tokens, k, cols)
    return {"dy": draw(tokens, cols, seed=16), **ops}, T.expert_combine_grad


def clip(*sizes, call=None):
    ops = {f"g{i}": draw(n, seed=17 + i) for i, n in enumerate(sizes)}

    def run(stream=None, **grads):
        grads = list(grads.values())
        if call:
            return call(grads, stream=stream)
        return (T.clip_grads(grads, 0.5, stream=stream), *grads)
    return ops, run


CASES = {
    "norm": lambda: norm(5, 300),
    "norm of long rows": lambda: norm(3, 40000),
    "norm of many rows": lambda: norm(1300, 1024),
    "norm of many odd rows": lambda: norm(3000, 1001),
    "norm to 8 bits": lambda: norm(1300, 1024, call=T.layernorm_fp8),
    "norm grad": lambda: norm_grad(5, 300),
    "norm grad of many rows": lambda: norm_grad(1300, 1024),
    "norm grad of odd rows": lambda: norm_grad(1300, 1001),
    "norm grad of long rows": lambda: norm_grad(170, 12296),
    "sort, one launch": lambda: sort(16, 4, 16),
    "sort, two launches": lambda: sort(16384, 8, 64),
    "sort, two launches, 32 bits": lambda: sort(20000, 4, 64, torch.int32),
    "sort, three launches": lambda: sort(16384, 8, 300),
    "dispatch": lambda: dispatch(900, 4, 520),
    "dispatch of odd rows": lambda: dispatch(900, 4, 133),
    "dispatch of many odd rows": lambda: dispatch(4000, 4, 1001),
    "dispatch of 8-bit rows": lambda: dispatch_fp8(900, 4, 512),
    "combine": lambda: combine(40, 3, 200),
    "combine of many rows": lambda: combine(5000, 4, 520),
    "combine of odd rows": lambda: combine(900, 4, 133),
    "combine grad": lambda: combine_grad(40, 3, 200),
    "combine grad of many rows": lambda: combine_grad(5000, 4, 520),
    "combine grad of odd rows": lambda: combine_grad(900, 4, 133),
    "grad norm": lambda: clip(3000, 77, call=T.grad_norm),
    "clip": lambda: clip(3000, 77),
    "clip of much": lambda: clip(12000003, 5000),
}


def other(t):
    """Other values that are as good as t's to a call."""
    if t.dtype in (torch.int32, torch.int64):
        return t.flip(0).roll(1, 1).contiguous()       # ids and slots: the same ones elsewhere
    if t.dtype == torch.float8_e4m3fn:
        return torch.zeros_like(t.view(torch.uint8)).view(t.dtype)
    return torch.full_like(t, 0.25)


def words(t):
    """A tensor's bytes as one row that expert_dispatch copies."""
    flat = t.reshape(-1)
    if t.dtype in (torch.int32, torch.int64):
        return flat.view(F32).view(1, -1)
    return flat.view(1, -1)


def raw(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def flat(r):
    return [t for t in (r if isinstance(r, (tuple, list)) else (r,)) if t is not None]


@pytest.mark.parametrize("by", ["copies", "calls"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_operands_that_are_still_being_written(name, by):
    true, call = CASES[name]()
    want = [raw(t).clone() for t in flat(call(**{n: t.clone() for n, t in true.items()}))]
    held = {n: other(t) for n, t in true.items()}
    first = [raw(t) for t in flat(call(**{n: t.clone() for n, t in held.items()}))]
    assert not all(torch.equal(u, v) for u, v in zip(first, want))     # the old values would show
    one = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    busy = torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(30):
            busy += 1
        for n, t in true.items():
            if by == "copies":
                raw(held[n]).copy_(raw(t))
            else:
                T.expert_dispatch(words(t), one, out=words(held[n]))
    got = flat(call(**held, stream=side))
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(raw(u), v) for u, v in zip(got, want))
