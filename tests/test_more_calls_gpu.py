"""GPU tests of the calls themselves (layer norm, routing, clipping): the compiled
calls take what they are meant to take and give what the Python way gives, bit
for bit; streams, memory pools, captured graphs and calls side by side."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import tile_size_decision_gb300 as T  # noqa: E402


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
    return [t for t in (r if isinstance(r, (tuple, list)) else (r,)) if t is not None]


def raw(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def cases(**kw):
    """Calls by name, each a function of no arguments, and each twice alike.  Rows that
    nobody names are zeros: outputs are given where there are such rows."""
    f32 = torch.float32
    x, r, w, b = draw(5, 300), draw(5, 300, seed=2), draw(300, seed=3), draw(300, seed=4)
    big, bigger = draw(900, 1024, seed=5), draw(900, 1024, seed=6)
    wb = draw(1024, seed=7)
    ids = torch.randint(0, 6, (40, 3), generator=torch.Generator().manual_seed(8)).cuda()
    many = torch.randint(-1, 60, (5000, 4), generator=torch.Generator().manual_seed(9)).cuda()
    slots, mslots = T.expert_sort(ids, 6)[0], T.expert_sort(many, 60)[0]
    t, rows = draw(40, 200, seed=10), draw(120, 200, seed=11)
    p, dy = draw(40, 3, dtype=f32, seed=12), draw(40, 200, seed=13)
    q, s = T.quantize_fp8(t)
    bt, brows, bp = draw(5000, 520, seed=14), draw(20000, 520, seed=15), draw(5000, 4, seed=16)
    grads = [draw(1000), draw(33, dtype=f32), draw(7, 9, dtype=torch.float16)]
    large = [draw(3000000, seed=17), draw(100001, dtype=f32, seed=18)]
    several = [draw(700 + i, seed=i) for i in range(300)]
    ring, odd = draw(1300, 4096, seed=19), draw(1300, 4001, seed=20)
    wr, wo = draw(4096, seed=21), draw(4001, seed=22)
    ot, orows = draw(5000, 133, seed=23), draw(20000, 133, seed=24)

    def for_call(t):
        """t, made on the current stream, for a call on the given one."""
        side = kw.get("stream")
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
            t.record_stream(side)
        return t

    def outs(*shape, dtype=torch.bfloat16):
        return for_call(torch.zeros(shape, dtype=dtype, device="cuda"))

    def like(ts):
        return [for_call(torch.zeros_like(t)) for t in ts]

    def clipped(ts, *args):
        out = like(ts)
        return [T.clip_grads(ts, *args, out=out, **kw), *out]

    def in_place(ts, *args):
        ts = [for_call(t.clone()) for t in ts]
        return [T.clip_grads(ts, *args, **kw), *ts]

    return {
        "norm": lambda: T.layernorm(x, w, **kw),
        "norm all": lambda: T.layernorm(x, w, b, residual=r, eps=1, **kw),
        "norm given": lambda: T.layernorm(x, w, b, residual=r, out=outs(5, 304)[:, 2:302],
                                          h_out=outs(5, 310)[:, :300], **kw),
        "norm parameter": lambda: T.layernorm(x, torch.nn.Parameter(w), **kw),
        "norm large": lambda: T.layernorm(big, wb, wb, residual=bigger, **kw),
        "norm many rows": lambda: T.layernorm(ring, wr, wr, residual=ring, **kw),
        "norm many odd rows": lambda: T.layernorm(odd, wo, wo, residual=odd, **kw),
        "norm fp8 many odd rows": lambda: T.layernorm_fp8(odd, wo, **kw),
        "norm fp8": lambda: T.layernorm_fp8(x, w, b, **kw),
        "norm fp8 large": lambda: T.layernorm_fp8(big, wb, residual=bigger, **kw),
        "norm fp8 given": lambda: T.layernorm_fp8(
            x, w, residual=r, out=outs(5, 300, dtype=torch.float8_e4m3fn),
            scales=outs(5, 3, dtype=f32), h_out=outs(5, 300), **kw),
        "norm of no rows": lambda: T.layernorm_fp8(x[:0], w, **kw),
        "norm grad": lambda: T.layernorm_grad(r, x, w, **kw),
        "norm grad large": lambda: T.layernorm_grad(big, bigger, wb, dh=big, **kw),
        "norm grad many odd rows": lambda: T.layernorm_grad(odd, odd, wo, dh=odd, **kw),
        "norm grad given": lambda: T.layernorm_grad(
            r, x, w, dh=x, dx_out=outs(5, 300), dweight_out=outs(300, dtype=f32),
            dbias_out=outs(300, dtype=f32), workspace=for_call(T.layernorm_grad_workspace(x)), **kw),
        "sort": lambda: T.expert_sort(ids, 6, **kw),
        "sort int32": lambda: T.expert_sort(ids.int()[:, 1:], 6, **kw),
        "sort many": lambda: T.expert_sort(many, 60, **kw),
        "sort of no rows": lambda: T.expert_sort(ids[:0], 6, **kw),
        "dispatch": lambda: T.expert_dispatch(t, slots, **kw),
        "dispatch large": lambda: T.expert_dispatch(bt, mslots, out=outs(20000, 520), **kw),
        "dispatch odd": lambda: T.expert_dispatch(ot, mslots, out=outs(20000, 133), **kw),
        "dispatch fp8": lambda: T.expert_dispatch(q, slots, scales=s, **kw),
        "dispatch fp8 given": lambda: T.expert_dispatch(
            q, slots, scales=s, out=outs(130, 200, dtype=torch.float8_e4m3fn),
            scales_out=outs(130, 2, dtype=f32), **kw),
        "combine": lambda: T.expert_combine(rows, slots, p, **kw),
        "combine plain": lambda: T.expert_combine(rows, slots, **kw),
        "combine large": lambda: T.expert_combine(brows, mslots, bp, **kw),
        "combine odd": lambda: T.expert_combine(orows, mslots, bp, **kw),
        "combine grad odd": lambda: T.expert_combine_grad(ot, orows, mslots, bp, drows_out=outs(20000, 133), **kw),
        "combine given": lambda: T.expert_combine(rows, slots, p.half(), out=outs(40, 210)[:, 3:203], **kw),
        "combine grad": lambda: T.expert_combine_grad(dy, rows, slots, p, **kw),
        "combine grad large": lambda: T.expert_combine_grad(
            bt, brows, mslots, bp, drows_out=outs(20000, 520), dweights_out=outs(5000, 4, dtype=f32), **kw),
        "grad norm": lambda: T.grad_norm(grads, **kw),
        "grad norm large": lambda: T.grad_norm(large, **kw),
        "clip": lambda: clipped(grads, 0.5),
        "clip large": lambda: clipped(large, 2, 0.0),
        "clip of 300": lambda: clipped(several, 0.5),
        "clip of 300 in place": lambda: in_place(several, 0.5),
        "clip in place": lambda: in_place(grads, 0.5),
        "clip large in place": lambda: in_place(large, 0.5),
    }


NAMES = sorted(cases())


@pytest.mark.parametrize("name", NAMES)
def test_the_compiled_calls_give_what_the_python_way_gives(name, counting, monkeypatch):
    call = cases()[name]
    before = counting.taken
    got = flat(call())
    assert counting.taken == before + 1
    monkeypatch.setattr(T, "_CALLS", T._NoCalls)
    want = flat(call())
    assert len(got) == len(want)
    for u, v in zip(got, want):
        assert u.dtype == v.dtype and u.shape == v.shape
        # (A single row's or column's stride means nothing.)
        assert [s for s, n in zip(u.stride(), u.shape) if n > 1] == \
            [s for s, n in zip(v.stride(), v.shape) if n > 1] or u.numel() == 0
        assert torch.equal(raw(u), raw(v))


def pool_of(t):
    """The stream whose pool holds t."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in any pool")


NEW = ["norm large", "norm fp8 large", "norm grad large", "sort many", "dispatch", "dispatch fp8", "combine",
       "combine grad", "grad norm large"]


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("name", NEW)
def test_outputs_on_a_given_stream_come_from_its_pool(name, compiled, monkeypatch):
    T._compiled()
    if not compiled:
        monkeypatch.setattr(T, "_CALLS", T._NoCalls)
    side = torch.cuda.Stream()
    want = flat(cases()[name]())
    call = cases(stream=side)[name]
    torch.cuda.synchronize()
    got = flat(call())
    side.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(raw(u), raw(v))
        assert pool_of(u) == side.cuda_stream
        assert pool_of(v) == torch.cuda.current_stream().cuda_stream
    assert torch.cuda.current_stream() != side


@pytest.mark.parametrize("name", NAMES)
def test_calls_on_a_side_stream_wait_for_its_work(name):
    # The stream is busy when the call comes: what it reads is written before.
    side = torch.cuda.Stream()
    want = flat(cases()[name]())
    call = cases(stream=side)[name]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy = torch.zeros(1 << 26, device="cuda")
        for _ in range(10):
            busy += 1
    got = flat(call())
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(raw(u), raw(v)) for u, v in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    call = cases()[name]
    want = [raw(t).clone() for t in flat(call())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    # Two graphs of the same call, replayed side by side: their scratch is their own.
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(flat(call()))
        graphs.append(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(raw(t), w) for t, w in zip(out, want))


def test_calls_side_by_side_on_two_streams():
    # Calls without a workspace of the caller's share nothing.
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    names = [n for n in NAMES if "in place" not in n and n not in ("clip", "clip large")]
    want = {n: [raw(t).clone() for t in flat(cases()[n]())] for n in names}
    on = {s: cases(stream=s) for s in (a, b)}
    torch.cuda.synchronize()
    got = {}
    for n in names:
        for s in (a, b):
            got[n, s] = [flat(on[s][n]()) for _ in range(3)]
    torch.cuda.synchronize()
    for (n, _), calls in got.items():
        for out in calls:
            assert all(torch.equal(raw(t), w) for t, w in zip(out, want[n])), n


def test_given_outputs_are_returned(counting):
    x, w = draw(5, 300), draw(300, seed=3)
    out, hh = torch.empty_like(x), torch.empty_like(x)
    y, h = T.layernorm(x, w, residual=x, out=out, h_out=hh)
    assert y is out and h is hh
    slots = torch.arange(10, dtype=torch.int32, device="cuda").view(5, 2)
    rows = torch.empty(10, 300, dtype=x.dtype, device="cuda")
    assert T.expert_dispatch(x, slots, out=rows) is rows
    assert T.expert_combine(rows, slots, out=out) is out
    dw = torch.empty(5, 2, device="cuda")
    p = torch.ones(5, 2, device="cuda")
    a, b = T.expert_combine_grad(x, rows, slots, p, drows_out=rows.clone(), dweights_out=dw)
    assert b is dw and counting.taken == 4


def test_a_lazy_list_of_gradients_and_autograd_leaves(counting):
    p = [torch.nn.Parameter(draw(30, dtype=torch.float32, seed=i)) for i in range(3)]
    sum((q * q).sum() for q in p).backward()
    before = [q.grad.clone() for q in p]
    norm = T.clip_grads((q.grad for q in p), 1.0)
    assert counting.taken == 1
    for q, g in zip(p, before):
        assert torch.allclose(q.grad, g / (norm + 1e-6), rtol=1e-6)
    # A parameter itself: its values change, not its history.
    v = p[0]._version
    T.clip_grads([p[0].data], 1e-3)
    assert p[0].requires_grad and p[0]._version >= v


def test_what_the_compiled_calls_refuse_is_named(counting):
    x, w = draw(5, 304), draw(304, seed=3)
    slots = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    for call, kind in [
        (lambda: T.layernorm(x.cpu(), w), ValueError),
        (lambda: T.layernorm(x[0], w), ValueError),
        (lambda: T.layernorm(x.t(), w), ValueError),
        (lambda: T.layernorm(x, w, w[:-1]), ValueError),
        (lambda: T.layernorm(x, w, w.float()), TypeError),
        (lambda: T.layernorm_fp8(x, w, scales=torch.zeros(5, 2, device="cuda")), ValueError),
        (lambda: T.layernorm_grad(x, x, w, dbias_out=w), TypeError),
        (lambda: T.layernorm_grad(x, x, w, workspace=torch.zeros(9, dtype=torch.uint8)), ValueError),
        (lambda: T.expert_sort(slots.float(), 4), TypeError),
        (lambda: T.expert_sort(slots, 0), T.TilesError),
        (lambda: T.expert_sort(slots, 5000), T.TilesError),
        (lambda: T.expert_sort(slots.t(), 4), ValueError),
        (lambda: T.expert_dispatch(x, slots.long()), TypeError),
        (lambda: T.expert_dispatch(x, slots[:4]), ValueError),
        (lambda: T.expert_dispatch(x, slots, out=x[:, :9]), ValueError),
        (lambda: T.expert_dispatch(x, slots, out=x[:1].expand(10, 304)), T.TilesError),
        (lambda: T.expert_combine(x, slots, x[:, :2].t()), ValueError),
        (lambda: T.expert_combine_grad(x, x, slots, None), Exception),
        (lambda: T.grad_norm([]), ValueError),
        (lambda: T.grad_norm([x, x.cpu()]), ValueError),
        (lambda: T.grad_norm([x[:, :9]]), ValueError),
        (lambda: T.grad_norm([slots]), TypeError),
        (lambda: T.clip_grads([x], float("nan")), T.TilesError),
        (lambda: T.clip_grads([x], 1.0, eps=-1.0), T.TilesError),
        (lambda: T.clip_grads([x, x], 1.0), T.TilesError),
        (lambda: T.clip_grads([x], 1.0, out=[w]), ValueError),
    ]:
        with pytest.raises(kind):
            call()
    assert counting.taken == 0
