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
