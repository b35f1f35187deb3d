"""GPU tests of a GEMM whose rows of C end inside 16 bytes, in a C whose row
pitch is longer: what lies behind a row is not C's and keeps its value.  The
products are those of integers, exact in fp32 (every partial sum is below 2^24)
and compared bit for bit after the one rounding to C's type."""

import numpy as np
import pytest

import synth_inputs as S
from oracle import gemm as OG

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402
from tests.gpu_util import TORCH_DT, to_cuda  # noqa: E402

VARIANTS = {(64, 1): 8, (128, 1): 6, (192, 1): 5, (256, 1): 4, (128, 2): 8, (256, 2): 6}
VARIANT_IDS = [f"bn{bn}_cg{cg}" for bn, cg in VARIANTS]
CANARY = 1536.0


def config(v, tail="auto"):
    bn, cg = v
    return T.make_config(128 * cg, bn, 64, VARIANTS[v], 192, "tcgen05", 2, cg, tail=tail)


def operands(m, n, k, dt, batch=None):
    lead = () if batch is None else (batch,)
    a, b = S.integer_matrix(5, (*lead, m, k), dt), S.integer_matrix(6, (*lead, k, n), dt)
    return a, b, to_cuda(a, dt, -(-k // 8) * 8), to_cuda(b, dt, -(-n // 8) * 8)


def expect(big, m, n, a, b, in_dt, out_dt):
    got = big.clone()
    view = got[..., :m, :n]
    want = torch.from_numpy(OG.gemm(S.widen(a, in_dt), S.widen(b, in_dt))) if a.ndim == 2 else \
        torch.from_numpy(np.stack([OG.gemm(S.widen(x, in_dt), S.widen(y, in_dt))
                                   for x, y in zip(a, b)]))
    assert torch.equal(view.cpu(), want.to(TORCH_DT[out_dt]))
    view.fill_(CANARY)
    assert bool((got == CANARY).all())


@pytest.mark.parametrize("v", list(VARIANTS), ids=VARIANT_IDS)
@pytest.mark.parametrize("out_dt", [S.F32, S.F16, S.BF16])
@pytest.mark.parametrize("short", [1, 2, 3, 5, 7])
def test_every_variant(v, out_dt, short):
    bn, cg = v
    m, n, k = 128 * cg + 37, 2 * bn + 40 - short, 72
    in_dt = S.BF16 if out_dt == S.BF16 else S.F16
    a, b, ta, tb = operands(m, n, k, in_dt)
    big = torch.full((m + 3, n + short + 16), CANARY, dtype=TORCH_DT[out_dt], device="cuda")
    ws = T.workspace()
    T.gemm(ta, tb, out=big[:m, :n], cfg=config(v), workspace=ws)
    T.check(ws)
    expect(big, m, n, a, b, in_dt, out_dt)


@pytest.mark.parametrize("n", [1, 3, 7, 31, 33, 63, 65, 127, 129, 257])
@pytest.mark.parametrize("out_dt", [S.F32, S.F16])
def test_narrow_and_batched(n, out_dt):
    batch, m, k = 3, 70, 72
    a, b, ta, tb = operands(m, n, k, S.F16, batch)
    pitch = -(-n // 8) * 8 + 8
    big = torch.full((batch, m + 2, pitch), CANARY, dtype=TORCH_DT[out_dt], device="cuda")
    ws = T.workspace()
    T.gemm_batched(ta, tb, out=big[:, :m, :n], workspace=ws)
    T.check(ws)
    expect(big, m, n, a, b, S.F16, out_dt)


@pytest.mark.parametrize("v", [(256, 2), (256, 1), (128, 1)], ids=["bn256_cg2", "bn256_cg1",
                                                                   "bn128_cg1"])
@pytest.mark.parametrize("out_dt", [S.F32, S.F16, S.BF16])
@pytest.mark.parametrize("tail", ["ksplit", "nhalf"])
@pytest.mark.parametrize("over", [0, 1])
def test_split_last_rounds(v, out_dt, tail, over):
    # One tile more than the first round takes: its last one is split along K or
    # into halves of its columns.  With `over` C has a second, narrow tile column.
    bn, cg = v
    groups = torch.cuda.get_device_properties(0).multi_processor_count // cg
    rows = groups + 1 if not over else groups // 2 + 1
    m, n, k = 128 * cg * rows - 37, bn - 43 + over * 100, 1000
    in_dt = S.BF16 if out_dt == S.BF16 else S.F16
    a, b, ta, tb = operands(m, n, k, in_dt)
    big = torch.full((m, -(-n // 8) * 8 + 16), CANARY, dtype=TORCH_DT[out_dt], device="cuda")
    c = big[:, :n]
    cfg = config(v, tail)
    ws = T.gemm_workspace(ta, tb, c, cfg)
    sch = T.gemm_schedule(ta, tb, c, cfg, ws)
    if not over:
        assert sch.tail_mode == (2 if tail == "ksplit" else 1)
    T.gemm(ta, tb, out=c, cfg=cfg, workspace=ws)
    T.check(ws)
    expect(big, m, n, a, b, in_dt, out_dt)
