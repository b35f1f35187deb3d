"""Arguments that the Python calls refuse before anything reaches the library (no GPU)."""

import pytest

torch = pytest.importorskip("torch")

import tile_size_decision_gb300 as T  # noqa: E402


class Stand:
    """What the checks look at of a CUDA tensor."""

    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_a_workspace_is_contiguous_and_on_the_gpu():
    assert T._workspace_args(None) == (None, 0)
    t = torch.zeros(256, dtype=torch.uint8)
    assert T._workspace_args(Stand(t)) == (t.data_ptr(), 256)
    with pytest.raises(ValueError, match="workspace"):
        T._workspace_args(t)
    # One byte that claims to be 256.
    with pytest.raises(ValueError, match="workspace"):
        T._workspace_args(Stand(torch.zeros(1, dtype=torch.uint8).expand(256)))


def test_the_calls_on_a_workspace_alone_refuse_it_too():
    t = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace"):
        T.check(t)
    with pytest.raises(ValueError, match="workspace"):
        T.selftest_wait_timeout(t, 1000)


def test_a_convolution_writes_to_the_gpu_only():
    x, w = Stand(torch.zeros(1, 4, 6, 6).half()), Stand(torch.zeros(4, 4, 3, 3).half())
    y = torch.zeros(1, 4, 4, 4).half()
    assert T._conv_desc(x, w, (1, 1), (0, 0), (1, 1), Stand(y), "nchw").y == y.data_ptr()
    with pytest.raises(ValueError, match="out"):
        T._conv_desc(x, w, (1, 1), (0, 0), (1, 1), y, "nchw")


class On(Stand):
    """A tensor on GPU `device`."""

    def __init__(self, device, *shape, dtype=torch.bfloat16):
        super().__init__(torch.zeros(shape, dtype=dtype))
        self.device_index = device

    def get_device(self):
        return self.device_index

    @property
    def device(self):
        return torch.device("cpu")          # where new outputs would go


E4M3 = torch.float8_e4m3fn


def operands(name, at):
    """A call's operands with the GPUs they are on, and the call."""
    def m(i, *shape, dtype=torch.bfloat16):
        return On(at[i % len(at)], *shape, dtype=dtype)

    f32, i32 = torch.float32, torch.int32
    return {
        "gemm": lambda: T.gemm(m(0, 4, 16), m(1, 16, 8), out=m(2, 4, 8)),
        "conv2d_htiled": lambda: T.conv2d_htiled(m(0, 1, 4, 6, 6), m(1, 4, 4, 3, 3),
                                                 out=m(2, 1, 4, 4, 4)),
        "rmsnorm": lambda: T.rmsnorm(m(0, 4, 16), m(1, 16), residual=m(2, 4, 16),
                                     out=m(3, 4, 16), h_out=m(4, 4, 16)),
        "rmsnorm_fp8": lambda: T.rmsnorm_fp8(m(0, 4, 16), m(1, 16), out=m(2, 4, 16, dtype=E4M3),
                                             scales=m(3, 4, 1, dtype=f32)),
        "rmsnorm_grad": lambda: T.rmsnorm_grad(
            m(0, 4, 16), m(1, 4, 16), m(2, 16), dh=m(3, 4, 16), dx_out=m(4, 4, 16),
            dweight_out=m(5, 16, dtype=f32)),
        "gemm_fp8": lambda: T.gemm_fp8(
            m(0, 4, 16, dtype=E4M3), m(1, 4, 1, dtype=f32), m(2, 8, 16, dtype=E4M3),
            m(3, 1, 1, dtype=f32), out=m(4, 4, 8)),
        "grouped_gemm_fp8": lambda: T.grouped_gemm_fp8(
            m(0, 4, 16, dtype=E4M3), m(1, 4, 1, dtype=f32), m(2, 2, 8, 16, dtype=E4M3),
            m(3, 2, 1, 1, dtype=f32), m(4, 3, dtype=i32), out=m(5, 4, 8)),
        "grouped_gemm": lambda: T.grouped_gemm(m(0, 4, 16), m(1, 2, 16, 8), m(2, 3, dtype=i32),
                                               out=m(3, 4, 8)),
        "grouped_wgrad": lambda: T.grouped_wgrad(m(0, 4, 16), m(1, 4, 8), m(2, 3, dtype=i32),
                                                 out=m(3, 2, 16, 8)),
        "workspace": lambda: T._workspace_args(m(0, 256, dtype=torch.uint8)),
    }[name]


@pytest.mark.parametrize("name", ["gemm", "conv2d_htiled", "rmsnorm", "rmsnorm_fp8",
                                  "rmsnorm_grad", "gemm_fp8", "grouped_gemm_fp8", "grouped_gemm",
                                  "grouped_wgrad", "workspace"])
def test_operands_of_another_gpu_are_refused(name, monkeypatch):
    class Library:
        """Stands in for the library: whatever reaches it was taken."""

        def __getattr__(self, name):
            def call(*args):
                raise AssertionError(f"{name} was called")
            return call

    monkeypatch.setattr(T, "conv_out_hw", lambda *a: (4, 4))
    monkeypatch.setattr(T, "_CALLS", T._NoCalls)
    monkeypatch.setattr(T, "load", Library)
    monkeypatch.setattr(T, "_raw_stream", lambda stream: 0)
    monkeypatch.setattr(T, "_stream_handle", lambda stream: None)
    monkeypatch.setattr(T, "_DEVICES", 2, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    if name != "workspace":
        with pytest.raises(AssertionError, match="was called"):
            operands(name, [0])()
    count = {"workspace": 1, "gemm": 3, "conv2d_htiled": 3, "rmsnorm_fp8": 4, "grouped_gemm": 4,
             "grouped_wgrad": 4, "rmsnorm": 5, "gemm_fp8": 5}.get(name, 6)
    for other in range(count):
        with pytest.raises(ValueError, match="current device"):
            operands(name, [1 if i == other else 0 for i in range(count)])()
    with pytest.raises(ValueError, match="current device"):
        operands(name, [1])()
