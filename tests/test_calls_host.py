"""Host-side checks of the compiled calls (no GPU): they are built and bound,
take nothing that is not on a GPU, and the Python functions then say so."""

import pytest

torch = pytest.importorskip("torch")

import tile_size_decision_gb300 as T  # noqa: E402
from tile_size_decision_gb300 import build  # noqa: E402


@pytest.fixture(scope="module")
def calls():
    build.build()
    return T._compiled()


def test_they_are_built_and_bound(calls):
    assert calls is not T._NoCalls
    for name in ("rmsnorm", "rmsnorm_grad", "product_fp8", "grouped_gemm", "grouped_wgrad"):
        assert callable(getattr(calls, name)) and hasattr(T._NoCalls, name)


def test_they_take_neither_host_tensors_nor_wrong_arguments(calls):
    x, w = torch.zeros(2, 16), torch.zeros(16)
    assert calls.rmsnorm(x, w, None, 1e-6, None, None, None, None, False) is None
    assert calls.rmsnorm(x, w) is None
    assert calls.rmsnorm(*[None] * 9) is None
    assert calls.rmsnorm_grad(x, x, w, "eps", None, None, None, None, None) is None
    assert calls.product_fp8(*[1] * 9) is None
    assert calls.grouped_gemm(x, x, x, False, None, None, None, None) is None
    assert calls.grouped_wgrad() is None
    with pytest.raises(TypeError):
        calls.bind(1, 2)


def test_the_functions_name_what_is_wrong(calls):
    x, w = torch.zeros(2, 16), torch.zeros(16)
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: T.rmsnorm(x, w), lambda: T.rmsnorm_fp8(x, w),
                 lambda: T.rmsnorm_grad(x, x, w), lambda: T.grouped_gemm(x, x[None], off),
                 lambda: T.grouped_wgrad(x, x, off)):
        with pytest.raises((ValueError, TypeError)):
            call()
