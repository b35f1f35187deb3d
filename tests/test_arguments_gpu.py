"""GPU tests of arguments that the Python calls refuse (nothing is launched)."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402


def calls(ws):
    """Every call that takes a workspace, by name, with this one."""
    x, w = torch.randn(20, 64, device="cuda").bfloat16(), torch.ones(64, device="cuda").bfloat16()
    b = torch.randn(3, 64, 40, device="cuda").bfloat16()
    off = torch.tensor([0, 4, 4, 20], dtype=torch.int32, device="cuda")
    x8, sx = T.quantize_fp8(x)
    w8, sw = T.quantize_fp8(b.transpose(1, 2).contiguous(), block_rows=128)
    img = torch.randn(1, 16, 8, 8, device="cuda").half()
    filt = torch.randn(16, 16, 3, 3, device="cuda").half()
    return {
        "gemm": lambda: T.gemm(x, b[0], workspace=ws),
        "gemm_batched": lambda: T.gemm_batched(x[None], b[:1], workspace=ws),
        "conv2d_htiled": lambda: T.conv2d_htiled(img, filt, workspace=ws),
        "conv2d_tiled": lambda: T.conv2d_tiled(img, filt, workspace=ws),
        "rmsnorm_grad": lambda: T.rmsnorm_grad(x, x, w, workspace=ws),
        "gemm_fp8": lambda: T.gemm_fp8(x8, sx, w8[0], sw[0], workspace=ws),
        "grouped_gemm_fp8": lambda: T.grouped_gemm_fp8(x8, sx, w8, sw, off, workspace=ws),
        "grouped_gemm": lambda: T.grouped_gemm(x, b, off, workspace=ws),
        "grouped_wgrad": lambda: T.grouped_wgrad(x, x, off, workspace=ws),
        "check": lambda: T.check(ws),
    }


def bad(kind):
    if kind == "host":
        return torch.zeros(1 << 20, dtype=torch.uint8)
    return torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 20)


@pytest.mark.parametrize("kind", ["host", "expanded"])
@pytest.mark.parametrize("name", ["gemm", "gemm_batched", "conv2d_htiled", "conv2d_tiled",
                                  "rmsnorm_grad", "gemm_fp8", "grouped_gemm_fp8", "grouped_gemm",
                                  "grouped_wgrad", "check"])
def test_a_workspace_on_the_host_or_smaller_than_it_says(name, kind):
    with pytest.raises(ValueError, match="workspace"):
        calls(bad(kind))[name]()
