"""GPU parity of the gradients' norm and clipping with the float64 definitions.

The squares of a thread's at most 64 elements are added in fp32, in at most 17
roundings of 2^-24; its sums of those lose nothing that counts; then come 5 levels
of lanes, 8 warps, a thread's share of the blocks' sums, 5 levels and 8 warps: under
60 roundings together, half of which reach the root, whose own argument and result
are rounded once more.  The norm is within 34 * 2^-24 of itself.  The factor adds its
own two roundings, a scaled element one fp32 product and half a spacing of its type."""

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
NAMES = {v: k for k, v in DT.items()}
REL = 36 * 2.0 ** -24


def draw(n, dtype, seed, scale=1.0, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n + shift, generator=g, device="cuda") * scale).to(DT[dtype])[shift:]


def f64(t):
    return t.double().cpu().numpy()


def assert_norm(got, grads):
    want = OO.clip([f64(g) for g in grads], 1.0)[0]
    assert got.shape == () and got.dtype == torch.float32 and got.is_cuda
    assert abs(float(got) - want) <= 34 * 2.0 ** -24 * want + 2.0 ** -149


def assert_clipped(got, grads64, types, max_norm, eps=1e-6):
    _, want = OO.clip(grads64, max_norm, eps)
    for g, w, t in zip(got, want, types):
        err = np.abs(f64(g) - w)
        tol = OT.ulp(w, NAMES[t]) / 2 * (1 + 2.0 ** -6) + 2 * REL * np.abs(w)
        assert np.all(err <= tol), f"worst error/tolerance {np.max(err / tol)}"


SETS = [
    [(1, "f32")], [(1, "bf16")], [(7, "f16")], [(8, "bf16")], [(2048, "bf16")], [(2049, "bf16")],
    [(4096, "f32"), (4095, "f32"), (1, "f32")],
    [(100000, "bf16"), (3, "f32"), (5000, "f16"), (0, "bf16"), (33, "bf16")],
    [(1500000, "f32"), (700001, "bf16")],
    [(12000003, "bf16"), (5, "f16"), (4096, "bf16"), (3000000, "f32")],
    [(n, ("f32", "bf16", "f16")[n % 3]) for n in range(1, 300)],       # three launches
]


@pytest.mark.parametrize("specs", SETS, ids=[str(len(s)) + "x" + str(s[0][0]) for s in SETS])
@pytest.mark.parametrize("given", [False, True])
def test_norm_and_clip(specs, given):
    grads = [draw(n, t, i, 0.1 + i % 3) for i, (n, t) in enumerate(specs)]
    before = [f64(g) for g in grads]
    types = [g.dtype for g in grads]
    assert_norm(T.grad_norm(grads), grads)
    max_norm = 0.25 * OO.clip(before, 1.0)[0]
    out = [torch.full_like(g, 7.0) for g in grads] if given else None
    norm = T.clip_grads(grads, max_norm, out=out)
    assert torch.equal(norm, T.grad_norm([torch.from_numpy(b).to(t).cuda()
                                          for b, t in zip(before, types)]))
    assert_clipped(out if given else grads, before, types, max_norm)
    if given:
        assert all(np.array_equal(f64(g), b) for g, b in zip(grads, before))


@pytest.mark.parametrize("given", [False, True])
def test_gradients_under_the_bound_stay_as_they_are(given):
    grads = [draw(5000, "bf16", 1), draw(3, "f32", 2)]
    before = [g.clone() for g in grads]
    out = [torch.zeros_like(g) for g in grads] if given else None
    norm = float(T.clip_grads(grads, 1e4, out=out))
    assert norm < 1e4
    for g, b in zip(out or grads, before):
        assert torch.equal(g, b)
    T.clip_grads(grads, float("inf"))
    assert all(torch.equal(g, b) for g, b in zip(grads, before))


@pytest.mark.parametrize("shift", [1, 3, 8])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_tensors_that_start_anywhere(shift, dtype):
    base = draw(70000 + 16, dtype, 3)
    g = base[shift:shift + 70000]
    edge = base[:shift].clone(), base[shift + 70000:].clone()
    before = f64(g)
    assert_norm(T.grad_norm([g]), [g])
    out = torch.zeros(70000 + 8, dtype=DT[dtype], device="cuda")
    T.clip_grads([g], 1.0, out=[out[8:]])                 # aligned apart
    assert_clipped([out[8:]], [before], [g.dtype], 1.0)
    assert not out[:8].any()
    T.clip_grads([g], 1.0)
    assert_clipped([g], [before], [g.dtype], 1.0)
    assert torch.equal(base[:shift], edge[0]) and torch.equal(base[shift + 70000:], edge[1])


def test_shapes_orders_and_one_tensor():
    g = draw(24000, "bf16", 4).view(20, 30, 40)
    for t in (g, g.permute(2, 0, 1), g[3:7], g[:, :1, :][:1]):
        assert_norm(T.grad_norm([t]), [t])
    assert torch.equal(T.grad_norm(g), T.grad_norm([g])) and torch.equal(T.grad_norm((g,)), T.grad_norm(iter([g])))
    before = f64(g)
    t = g.permute(1, 2, 0)
    out = torch.empty_like(t)                             # the same order of elements
    T.clip_grads([t], 2.0, out=[out])
    assert_clipped([out.permute(2, 0, 1)], [before], [g.dtype], 2.0)
    with pytest.raises(ValueError, match="together"):
        T.grad_norm([g[:, ::2]])
    with pytest.raises(ValueError, match="strides"):
        T.clip_grads([t], 2.0, out=[torch.empty(t.shape, dtype=t.dtype, device="cuda")])
    p = torch.nn.Parameter(torch.ones(8, device="cuda"))
    assert float(T.grad_norm([p])) == pytest.approx(8 ** 0.5, rel=1e-6)


def test_numbers_whose_squares_leave_the_range():
    for scale in (1e30, 1e-30, 1e-42):                    # over, under, denormal
        for n in (1, 5000, 3000000):
            g = draw(n, "f32", 5, scale)
            assert_norm(T.grad_norm([g]), [g])
    big, small = draw(4000, "bf16", 6, 1e25), draw(4000, "f32", 7, 1e-25)
    assert_norm(T.grad_norm([big, small]), [big, small])
    assert_norm(T.grad_norm([small, torch.zeros(9, device="cuda")]), [small])
    before = f64(big)
    T.clip_grads([big], 1.0)
    assert_clipped([big], [before], [big.dtype], 1.0)
    # 3e38 a piece: the norm is past fp32's range.
    assert float(T.grad_norm([torch.full((100,), 3e38, device="cuda")])) == float("inf")


def test_zeros_infinities_and_nans():
    z = torch.zeros(5000, device="cuda")
    assert float(T.grad_norm([z])) == 0 and float(T.clip_grads([z], 0.0, eps=0.0)) == 0
    assert not z.any()
    for n in (10, 3000000):
        g = draw(n, "bf16", 8)
        g[3] = float("inf")
        other = draw(100, "f32", 9)
        assert float(T.clip_grads([g, other], 1.0)) == float("inf")
        assert bool(g[3].isnan()) and int(g.isnan().sum()) == 1 and not other.any()
        g = draw(n, "f16", 8)
        g[n // 2] = float("nan")
        assert torch.isnan(T.clip_grads([g, other], 1.0))
        assert bool(g.isnan().all()) and bool(other.isnan().all())


def test_no_elements():
    e = torch.empty(0, device="cuda")
    assert float(T.grad_norm([e])) == 0 and float(T.clip_grads([e, e], 1.0)) == 0


def test_many_tensors_and_a_given_workspace():
    grads = [draw(1 + 37 * i % 501, "bf16", i) for i in range(1000)]
    before = [f64(g) for g in grads]
    n = T.load().tiles_grad_norm_workspace_bytes(1000)
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
    norm = T.clip_grads(grads, 3.0, workspace=ws)
    assert abs(float(norm) - OO.clip(before, 3.0)[0]) <= REL * float(norm)
    assert_clipped(grads, before, [g.dtype for g in grads], 3.0)
    assert bool((ws[:256] == 255).all()) and bool((ws[n:] == 255).all())
    with pytest.raises(T.TilesError, match="workspace"):
        T.grad_norm(grads, workspace=ws[:4096])


def test_overlapping_tensors_are_refused():
    g = draw(100, "f32", 10)
    for grads, out in (([g, g], None), ([g, g[50:]], None), ([g[:50], g[50:]], [g[50:], g[:50]]),
                       ([g[:50]], [g[1:51]])):
        with pytest.raises(T.TilesError, match="overlap"):
            T.clip_grads(grads, 1.0, out=out)
    # The norm alone only reads: a tensor given twice counts twice.
    assert_norm(T.grad_norm([g, g]), [g, g])
    # Its own gradient as the output is in place.
    before = f64(g)
    T.clip_grads([g], 1.0, out=[g])
    assert_clipped([g], [before], [g.dtype], 1.0)


def test_repeated_calls_give_the_same_bits():
    grads = [draw(3000000, "bf16", 11), draw(1000001, "f32", 12)]
    first = T.grad_norm(grads)
    out = [torch.empty_like(g) for g in grads]
    for _ in range(4):
        assert torch.equal(T.grad_norm(grads), first)
        assert torch.equal(T.clip_grads(grads, 1.0, out=out), first)
