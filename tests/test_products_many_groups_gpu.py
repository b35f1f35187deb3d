"""GPU parity of the grouped products with many groups, at the tolerances of
test_products_gpu (derived there): few rows spread over them, and enough
rows for the kernels on CTA pairs."""

import numpy as np
import pytest

from oracle import operators as OO
from oracle import tolerance as OT

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402


def f64(t):
    return t.double().cpu().numpy()


def draw(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def spread_rows(rows, groups, seed):
    """Offsets of `rows` rows that each pick a group; some are left out."""
    rng = np.random.default_rng(seed)
    counts = np.bincount(rng.integers(0, groups, rows) // 2 * 2, minlength=groups)
    off = np.concatenate([[0], np.cumsum(counts)])
    return off, torch.tensor(off, dtype=torch.int32, device="cuda")


def assert_close(got, ref, bound, dtype, rel):
    ok, worst, idx = OT.check(f64(got), ref, bound, dtype, rel)
    assert ok, f"worst error/tolerance {worst} at {idx}"


# Few rows: the contraction is split over a cluster.  Many: tiles on CTA pairs.
@pytest.mark.parametrize("rows,groups,n,k", [
    (1, 32, 136, 4096), (1, 256, 512, 2048), (3, 70, 256, 1024), (16, 256, 136, 2048),
    (9000, 70, 256, 192), (20000, 256, 264, 128), (12000, 129, 512, 64),
    (20000, 4096, 136, 64)])
@pytest.mark.parametrize("kind", ["16 bits", "transposed", "8 bits"])
def test_products(rows, groups, n, k, kind):
    off, toff = spread_rows(rows, groups, groups)
    ws = T.workspace()
    if kind == "8 bits":
        a, sa = T.quantize_fp8(draw((rows, k), 1))
        b, sb = T.quantize_fp8(draw((groups, n, k), 2), block_rows=128)
        c = T.grouped_gemm_fp8(a, sa, b, sb, toff, out_dtype="f32", workspace=ws)
        T.check(ws)
        ref, bound = OO.grouped_fp8(f64(a), f64(sa), f64(b), f64(sb), off)
        rel = (4 + OO.blocks(k) + 8) * 2.0 ** -22
    else:
        trans = kind == "transposed"
        a = draw((rows, k), 3).bfloat16()
        b = draw((groups, n, k) if trans else (groups, k, n), 4).bfloat16()
        c = T.grouped_gemm(a, b, toff, trans_b=trans, out_dtype="f32", workspace=ws)
        T.check(ws)
        ref, bound = OO.grouped(f64(a), f64(b), off, trans_b=trans)
        rel = ((k + 15) // 16 + 8) * 2.0 ** -22
    assert_close(c, ref, bound, "f32", rel)


@pytest.mark.parametrize("rows,groups,n,k", [(9000, 70, 256, 192), (500, 256, 72, 136)])
def test_weight_gradients(rows, groups, n, k):
    off, toff = spread_rows(rows, groups, groups + 1)
    ws = T.workspace()
    a, dc = draw((rows, k), 5).bfloat16(), draw((rows, n), 6).bfloat16()
    dw = T.grouped_wgrad(a, dc, toff, out_dtype="f32", workspace=ws)
    T.check(ws)
    ref, bound = OO.wgrad(f64(a), f64(dc), off)
    steps = (int(np.max(np.diff(off))) + 15) // 16
    assert_close(dw, ref, bound, "f32", (steps + 8) * 2.0 ** -22)
