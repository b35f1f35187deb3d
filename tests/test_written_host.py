"""The Python way of the calls raises the versions of the tensors that they are given to
write, and of no others (no GPU: the library that launches is a stand-in)."""

import pytest

torch = pytest.importorskip("torch")

import tile_size_decision_gb300 as T  # noqa: E402

F32, I32, E4M3 = torch.float32, torch.int32, torch.float8_e4m3fn


class OnGpu(torch.Tensor):
    """A tensor of the host that says it is on a GPU."""

    @property
    def is_cuda(self):
        return True


def m(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Library:
    def __getattr__(self, name):
        return lambda *args: 256 if name.endswith("workspace_bytes") else 0


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    monkeypatch.setattr(T, "_CALLS", T._NoCalls)
    monkeypatch.setattr(T, "load", Library)
    monkeypatch.setattr(T, "_raw_stream", lambda stream: 0)
    monkeypatch.setattr(T, "_DEVICES", 1, raising=False)


def calls():
    """By name: what a call reads, what it writes, and the call."""
    x, r, w, b, o, h = m(4, 16), m(4, 16), m(16), m(16), m(4, 16), m(4, 16)
    o8, s, s2 = m(4, 16, dtype=E4M3), m(4, 1, dtype=F32), m(8, 1, dtype=F32)
    dw, db = m(16, dtype=F32), m(16, dtype=F32)
    slots, p, dp = m(4, 2, dtype=I32), m(4, 2, dtype=F32), m(4, 2, dtype=F32)
    rows, more = m(8, 16), m(8, 16)
    g, to = [m(4, 16), m(3, dtype=F32)], [m(4, 16), m(3, dtype=F32)]
    return {
        "layernorm": ([x, w, b, r], [o, h], lambda: T.layernorm(x, w, b, residual=r, out=o, h_out=h)),
        "layernorm in place": ([x, w], [r], lambda: T.layernorm(x, w, residual=r, h_out=r)),
        "layernorm_fp8": ([x, w], [o8, s], lambda: T.layernorm_fp8(x, w, out=o8, scales=s)),
        "layernorm_grad": ([x, h, w, r], [o, dw, db], lambda: T.layernorm_grad(
            x, h, w, dh=r, dx_out=o, dweight_out=dw, dbias_out=db)),
        "expert_dispatch": ([x, slots, s], [more, s2], lambda: T.expert_dispatch(
            x, slots, scales=s, out=more, scales_out=s2)),
        "expert_combine": ([rows, slots, p], [o], lambda: T.expert_combine(rows, slots, p, out=o)),
        "expert_combine_grad": ([x, rows, slots, p], [more, dp], lambda: T.expert_combine_grad(
            x, rows, slots, p, drows_out=more, dweights_out=dp)),
        "grad_norm": (g, [], lambda: T.grad_norm(g)),
        "clip_grads": ([], g, lambda: T.clip_grads(g, 1.0)),
        "clip_grads apart": (g, to, lambda: T.clip_grads(g, 1.0, out=to)),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_versions(name):
    read, written, call = calls()[name]
    was = [t._version for t in read], [t._version for t in written]
    call()
    assert [t._version for t in read] == was[0]
    assert all(t._version > v for t, v in zip(written, was[1]))


@pytest.mark.parametrize("name", sorted(calls()))
def test_tensors_without_a_version(name):
    with torch.inference_mode():
        _, _, call = calls()[name]
        call()
    call()
