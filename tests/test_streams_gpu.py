"""New outputs of a call on a given stream come from that stream's pool: memory
of the current stream's pool may still be in use by work pending there."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402


def pool_of(t):
    """The stream whose pool holds t."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in any pool")


def norms(**kw):
    x, w = torch.randn(700, 1024, device="cuda").bfloat16(), torch.ones(1024, device="cuda")
    g = T.rmsnorm_grad_workspace(x)
    return {
        "rmsnorm": lambda: T.rmsnorm(x, w, residual=x, **kw),
        "rmsnorm_fp8": lambda: T.rmsnorm_fp8(x, w, residual=x, **kw),
        "rmsnorm_grad": lambda: T.rmsnorm_grad(x, x, w, workspace=g, **kw),
        "quantize_fp8": lambda: T.quantize_fp8(x, **kw),
        "quantize_fp8 blocks": lambda: T.quantize_fp8(x, block_rows=128, **kw),
    }


def products(**kw):
    ws = T.workspace()
    a, b = torch.randn(700, 256, device="cuda").bfloat16(), torch.randn(3, 256, 512, device="cuda").bfloat16()
    dc = torch.randn(700, 512, device="cuda").bfloat16()
    off = torch.tensor([0, 200, 200, 700], dtype=torch.int32, device="cuda")
    a8, sa = T.quantize_fp8(a)
    b8, sb = T.quantize_fp8(b.transpose(1, 2).contiguous(), block_rows=128)
    return {
        "gemm_fp8": lambda: T.gemm_fp8(a8, sa, b8[0], sb[0], workspace=ws, **kw),
        "grouped_gemm_fp8": lambda: T.grouped_gemm_fp8(a8, sa, b8, sb, off, workspace=ws, **kw),
        "grouped_gemm": lambda: T.grouped_gemm(a, b, off, workspace=ws, **kw),
        "grouped_wgrad": lambda: T.grouped_wgrad(a, dc, off, workspace=ws, **kw),
    }


def outputs(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


def check(build, name):
    side = torch.cuda.Stream()
    want = outputs(build()[name]())
    call = build(stream=side)[name]
    torch.cuda.synchronize()
    got = outputs(call())
    side.synchronize()
    for u, v in zip(got, want):
        assert pool_of(u) == side.cuda_stream
        assert pool_of(v) == torch.cuda.current_stream().cuda_stream
        assert u.shape == v.shape and u.dtype == v.dtype
    assert torch.cuda.current_stream() != side
    # The stream named is the default one, the current one is not.
    with torch.cuda.stream(side):
        call = build(stream=torch.cuda.default_stream())[name]
        torch.cuda.synchronize()
        for t in outputs(call()):
            assert pool_of(t) == torch.cuda.default_stream().cuda_stream
        assert torch.cuda.current_stream() == side
    torch.cuda.synchronize()


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("name", ["rmsnorm", "rmsnorm_fp8", "rmsnorm_grad", "quantize_fp8",
                                  "quantize_fp8 blocks"])
def test_norms(name, compiled, monkeypatch):
    T._compiled()
    if not compiled:
        monkeypatch.setattr(T, "_CALLS", T._NoCalls)
    check(norms, name)


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("name", ["gemm_fp8", "grouped_gemm_fp8", "grouped_gemm", "grouped_wgrad"])
def test_products(name, compiled, monkeypatch):
    T._compiled()
    if not compiled:
        monkeypatch.setattr(T, "_CALLS", T._NoCalls)
    check(products, name)


def matmuls(**kw):
    ws = T.workspace()
    a, b = torch.randn(256, 128, device="cuda").half(), torch.randn(128, 512, device="cuda").half()
    x, w = torch.randn(2, 16, 20, 20, device="cuda").half(), torch.randn(32, 16, 3, 3, device="cuda").half()
    return {
        "gemm": lambda: T.gemm(a, b, workspace=ws, **kw),
        "gemm_batched": lambda: T.gemm_batched(a[None], b[None], workspace=ws, **kw),
        "gemm_noalloc": lambda: T.gemm_noalloc(a[None], b[None], **kw),
        "conv2d_htiled": lambda: T.conv2d_htiled(x, w, workspace=ws, **kw),
        "conv2d_tiled": lambda: T.conv2d_tiled(x, w, workspace=ws, **kw),
    }


@pytest.mark.parametrize("name", ["gemm", "gemm_batched", "gemm_noalloc", "conv2d_htiled",
                                  "conv2d_tiled"])
def test_matrix_products_and_convolutions(name):
    check(matmuls, name)
