"""GPU tests of the compiled calls: they take what they are meant to take (no
silent way round them), and give what the Python way gives, bit for bit."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402

NAMES = ("rmsnorm", "rmsnorm_grad", "product_fp8", "grouped_gemm", "grouped_wgrad")


class Counting:
    """The compiled calls, counting those that they took."""

    def __init__(self, calls):
        self.calls, self.taken = calls, 0

    def __getattr__(self, name):
        fn = getattr(self.calls, name)

        def call(*args):
            r = fn(*args)
            self.taken += r is not None
            return r
        return call


@pytest.fixture()
def counting(monkeypatch):
    T._compiled()
    assert T._CALLS is not T._NoCalls
    c = Counting(T._CALLS)
    monkeypatch.setattr(T, "_CALLS", c)
    return c


def draw(*shape, dtype=torch.bfloat16, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


def cases():
    """Calls by name, each a function of no arguments, and each twice alike."""
    ws = T.workspace()
    x, r, w = draw(5, 300), draw(5, 300, seed=2), draw(300, seed=3)
    x32, w32 = draw(5, 300, dtype=torch.float32), draw(300, dtype=torch.float32)
    one = draw(1, 300, seed=4)
    a, b = draw(20, 64, seed=5), draw(3, 64, 40, seed=6)
    off = torch.tensor([0, 4, 4, 20], dtype=torch.int32, device="cuda")
    bt = b.transpose(1, 2).contiguous()
    dc = draw(20, 40, seed=7)
    a8, sa = T.quantize_fp8(draw(20, 300, seed=8))
    b8, sb = T.quantize_fp8(draw(200, 300, seed=9), block_rows=128)
    g8, sg = T.quantize_fp8(draw(3, 200, 300, seed=10), block_rows=128)
    gws = T.rmsnorm_grad_workspace(x)

    def outs(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    return {
        "norm": lambda: T.rmsnorm(x, w),
        "norm eps": lambda: T.rmsnorm(x, w, eps=1),
        "norm residual": lambda: T.rmsnorm(x, w, residual=r),
        "norm given": lambda: T.rmsnorm(x, w, residual=r, out=outs(5, 304)[:, 2:302],
                                        h_out=outs(5, 310)[:, :300]),
        "norm f32": lambda: T.rmsnorm(x32, w, residual=x32),
        "norm parameter": lambda: T.rmsnorm(x, torch.nn.Parameter(w32)),
        "norm one row": lambda: T.rmsnorm_fp8(one, w, residual=one),
        "norm fp8": lambda: T.rmsnorm_fp8(x, w),
        "norm fp8 given": lambda: T.rmsnorm_fp8(
            x, w, residual=r, out=outs(5, 300, dtype=torch.float8_e4m3fn),
            scales=outs(5, 3, dtype=torch.float32), h_out=outs(5, 300)),
        "norm of no rows": lambda: T.rmsnorm_fp8(x[:0], w),
        "norm grad": lambda: T.rmsnorm_grad(r, x, w, workspace=gws),
        "norm grad given": lambda: T.rmsnorm_grad(
            r, x, w, dh=x, dx_out=outs(5, 300), dweight_out=outs(300, dtype=torch.float32),
            workspace=gws),
        "fp8": lambda: T.gemm_fp8(a8, sa, b8, sb, workspace=ws),
        "fp8 f32": lambda: T.gemm_fp8(a8, sa, b8, sb, out_dtype="f32", workspace=ws),
        "fp8 torch type": lambda: T.gemm_fp8(a8, sa, b8, sb, out_dtype=torch.float16, workspace=ws),
        "fp8 given": lambda: T.gemm_fp8(a8, sa, b8, sb, out=outs(20, 210)[:, 1:201], workspace=ws),
        "fp8 one row": lambda: T.gemm_fp8(a8[3:4], sa[3:4], b8, sb, workspace=ws),
        "grouped fp8": lambda: T.grouped_gemm_fp8(a8, sa, g8, sg, off, workspace=ws),
        "grouped": lambda: T.grouped_gemm(a, b, off, workspace=ws),
        "grouped f32": lambda: T.grouped_gemm(a, b, off, out_dtype="f32", workspace=ws),
        "grouped trans": lambda: T.grouped_gemm(a, bt, off, trans_b=True, workspace=ws),
        "grouped given": lambda: T.grouped_gemm(a, b, off, out=outs(20, 48)[:, :40], workspace=ws),
        "wgrad": lambda: T.grouped_wgrad(a, dc, off, workspace=ws),
        "wgrad given": lambda: T.grouped_wgrad(a, dc, off, out=outs(3, 65, 41)[:, :64, :40],
                                               workspace=ws),
    }


def test_the_compiled_calls_give_what_the_python_way_gives(counting, monkeypatch):
    for name, call in cases().items():
        before = counting.taken
        got = flat(call())
        assert counting.taken == before + 1, name
        monkeypatch.setattr(T, "_CALLS", T._NoCalls)
        want = flat(call())
        monkeypatch.setattr(T, "_CALLS", counting)
        assert len(got) == len(want)
        for u, v in zip(got, want):
            assert u.dtype == v.dtype and u.shape == v.shape, name
            # (A single row's or column's stride means nothing.)
            assert [s for s, n in zip(u.stride(), u.shape) if n > 1] == \
                [s for s, n in zip(v.stride(), v.shape) if n > 1] or u.numel() == 0, name
            assert torch.equal(u.view(torch.uint8) if u.dtype == torch.float8_e4m3fn else u,
                               v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v), name


def test_the_compiled_calls_keep_given_outputs_and_the_input(counting):
    x, w = draw(5, 300), draw(300, seed=3)
    y, h = T.rmsnorm(x, w)
    assert h is x
    out, hh = torch.empty_like(x), torch.empty_like(x)
    y, h = T.rmsnorm(x, w, residual=x, out=out, h_out=hh)
    assert y is out and h is hh and counting.taken == 2


def test_the_compiled_calls_run_on_the_given_and_on_the_current_stream(counting):
    x, w = draw(2000, 4096), draw(4096, seed=3)
    want, _ = T.rmsnorm(x, w)
    for given in (True, False):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            late = x + 0
            for _ in range(20):
                late = late + 0
            if not given:
                got, _ = T.rmsnorm(late, w)
        if given:
            got, _ = T.rmsnorm(late, w, stream=side)
        side.synchronize()
        assert torch.equal(got, want)


def test_what_the_compiled_calls_refuse_is_named(counting):
    ws = T.workspace()
    x, w = draw(5, 304), draw(304, seed=3)
    a, b = draw(20, 64), draw(3, 64, 40)
    off = torch.tensor([0, 4, 4, 20], dtype=torch.int32, device="cuda")
    for call, kind in [
        (lambda: T.rmsnorm(x.cpu(), w), ValueError),
        (lambda: T.rmsnorm(x[0], w), ValueError),
        (lambda: T.rmsnorm(x.t(), w), ValueError),
        (lambda: T.rmsnorm(x, w[:-1]), ValueError),
        (lambda: T.rmsnorm(x, w, residual=x.half()), TypeError),
        (lambda: T.rmsnorm(x.double(), w), TypeError),
        (lambda: T.rmsnorm_fp8(x, w, scales=torch.zeros(5, 2, device="cuda")), ValueError),
        (lambda: T.rmsnorm_grad(x, x, w), T.TilesError),
        (lambda: T.grouped_gemm(a, b, off), T.TilesError),
        (lambda: T.grouped_gemm(a, b, off.cpu(), workspace=ws), ValueError),
        (lambda: T.grouped_gemm(a, b, off, out_dtype=torch.int32, workspace=ws), Exception),
        (lambda: T.grouped_gemm(a, b.half(), off, workspace=ws), TypeError),
        (lambda: T.grouped_wgrad(a, a[:5], off, workspace=ws), ValueError),
    ]:
        with pytest.raises(kind):
            call()
    assert counting.taken == 0
