"""tile_size_decision_gb300 — constraint-planned tiled GEMM and H-tiled
convolution for NVIDIA GB300 (sm_103a), with the norms, 8-bit products and
expert-grouped products that surround the GEMM in a transformer block.

A thin Python binding over libtiles.so (C ABI in include/tiles.h).  The
binding only marshals arguments: planning (C0-C4), tensor-map encoding and
every kernel run in the native library.  PyTorch supplies device memory and
streams.  Names follow the C ABI without the ``tiles_`` prefix.
"""

from __future__ import annotations

import contextlib
import ctypes as C
import os
import struct
import warnings

from . import _abi
from ._abi import TilesError, check as _check

__all__ = [
    "TilesError", "load", "version", "device_preset", "device_query", "evaluate",
    "finish_parallelism", "c0_bytes", "plan", "htile_rows", "workspace_bytes", "workspace",
    "gemm_variants", "gemm_variant_info",
    "gemm", "gemm_batched", "gemm_schedule", "gemm_workspace", "gemm_noalloc", "gemm_autotune",
    "gemm_host", "conv2d_host",
    "tuned_lookup", "tuned_save", "tuned_load", "tuned_clear", "conv2d_htiled", "conv2d_tiled",
    "conv_workspace",
    "conv_out_shape", "conv_out_hw", "check", "selftest_wait_timeout", "selftest_drop_stage",
    "make_config",
    "rmsnorm", "rmsnorm_fp8", "rmsnorm_grad", "rmsnorm_grad_workspace", "quantize_fp8",
    "gemm_fp8", "grouped_gemm", "grouped_gemm_fp8", "grouped_wgrad",
]


def load():
    return _abi.load()


def version() -> str:
    return load().tiles_version().decode()


def device_preset(name: str = "gb300") -> _abi.Device:
    d = _abi.Device()
    pid = {"h100_pages": _abi.DEV_H100_PAGES, "gb300": _abi.DEV_GB300}[name]
    _check(load().tiles_device_preset(pid, C.byref(d)), "tiles_device_preset")
    return d


def device_query(ordinal: int = 0) -> _abi.Device:
    d = _abi.Device()
    _check(load().tiles_device_query(ordinal, C.byref(d)), "tiles_device_query")
    return d


CONV_WEIGHTS = {"auto": _abi.CONV_W_AUTO, "smem": _abi.CONV_W_SMEM, "tmem": _abi.CONV_W_TMEM,
                "rows": _abi.CONV_W_TMEM_ROWS, "rows_direct": _abi.CONV_W_TMEM_ROWS_DIRECT}
TAILS = {"auto": _abi.TAIL_AUTO, "whole": _abi.TAIL_WHOLE, "nhalf": _abi.TAIL_NHALF,
         "ksplit": _abi.TAIL_KSPLIT}


def make_config(bm, bn, bk, stages=3, threads=128, instr="wgmma", acc_bufs=0,
                cta_group=0, tail="auto", conv_weights="auto") -> _abi.Config:
    c = _abi.Config()
    c.bm, c.bn, c.bk, c.stages, c.threads = bm, bn, bk, stages, threads
    c.instr = _abi.INSTR_CODES[instr] if isinstance(instr, str) else instr
    c.acc_bufs, c.cta_group = acc_bufs, cta_group
    c.tail = TAILS[tail] if isinstance(tail, str) else tail
    c.conv_weights = CONV_WEIGHTS[conv_weights] if isinstance(conv_weights, str) else conv_weights
    return c


def evaluate(dev: _abi.Device, cfg: _abi.Config, elem_bytes: int = 2,
             accum_bytes: int = 4) -> _abi.Verdict:
    v = _abi.Verdict()
    _check(load().tiles_evaluate(C.byref(dev), C.byref(cfg), elem_bytes, accum_bytes,
                                 C.byref(v)), "tiles_evaluate")
    return v


def finish_parallelism(dev: _abi.Device, v: _abi.Verdict, m: int, n: int,
                       b: int = 1) -> _abi.Verdict:
    _check(load().tiles_finish_parallelism(C.byref(dev), b, m, n, C.byref(v)),
           "tiles_finish_parallelism")
    return v


def c0_bytes(m, n, k, bm, bn, in_bytes=2, out_bytes=None, b=1) -> float:
    if out_bytes is None:
        out_bytes = in_bytes
    return load().tiles_c0_bytes(b, m, n, k, bm, bn, in_bytes, out_bytes)


def plan(m: int, n: int, k: int, b: int = 1, in_dtype: str = "f16", out_dtype: str | None = None,
         mode: str = "gb300", instr: str = "tcgen05", device: _abi.Device | None = None,
         capacity: int | None = None):
    """Ranked feasible verdicts (best first) and the count of feasible ones."""
    lib = load()
    if device is None:
        device = device_preset("gb300" if mode == "gb300" else "h100_pages")
    p = _abi.Problem()
    p.b, p.m, p.n, p.k = b, m, n, k
    p.in_dtype = _abi.DTYPE_CODES[in_dtype]
    p.out_dtype = _abi.DTYPE_CODES[out_dtype or in_dtype]
    p.instr = _abi.INSTR_CODES[instr]
    p.mode = {"pages": _abi.MODE_PAGES, "gb300": _abi.MODE_GB300}[mode]
    nf = C.c_int(0)
    _check(lib.tiles_plan(C.byref(device), C.byref(p), None, 0, C.byref(nf)), "tiles_plan")
    cap = nf.value if capacity is None else min(capacity, nf.value)
    out = (_abi.Verdict * max(cap, 1))()
    _check(lib.tiles_plan(C.byref(device), C.byref(p), out, cap, C.byref(nf)), "tiles_plan")
    return list(out[:cap]), nf.value


def gemm_variants() -> list:
    """The compiled GEMM kernel variants as configurations (no GPU needed)."""
    lib = load()
    out = []
    for i in range(lib.tiles_gemm_variant_count()):
        c = _abi.Config()
        _check(lib.tiles_gemm_variant(i, C.byref(c)), "tiles_gemm_variant")
        out.append(c)
    return out


def gemm_variant_info(index: int) -> _abi.VariantInfo:
    """What the CUDA runtime reports for compiled variant `index` on the
    current device: registers, shared memory, resident blocks and groups."""
    info = _abi.VariantInfo()
    _check(load().tiles_gemm_variant_info(index, C.byref(info)), "tiles_gemm_variant_info")
    return info


def htile_rows(H, kh, sh, pt, d, o0, o1) -> _abi.HTile:
    t = _abi.HTile()
    _check(load().tiles_htile_rows(H, kh, sh, pt, d, o0, o1, C.byref(t)), "tiles_htile_rows")
    return t


def workspace_bytes() -> int:
    return int(load().tiles_workspace_bytes())


# ---- kernels (need torch and a GPU) --------------------------------------------


_TORCH = None
_DTYPE_CODES = None
_RAW_STREAM = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _dtype_code(t) -> int:
    global _DTYPE_CODES
    if _DTYPE_CODES is None:
        torch = _torch()
        _DTYPE_CODES = {torch.float16: _abi.F16, torch.bfloat16: _abi.BF16,
                        torch.float32: _abi.F32}
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _stream_handle(stream):
    """The CUDA stream handle of `stream`, or of the current device's current
    stream.  The latter is read through torch's raw-stream query where it
    exists (torch.cuda.current_stream() builds a Python object per call)."""
    global _RAW_STREAM
    if stream is not None:
        return C.c_void_p(stream.cuda_stream)
    if _RAW_STREAM is None:
        tc = _torch()._C
        if hasattr(tc, "_cuda_getCurrentRawStream") and hasattr(tc, "_cuda_getDevice"):
            get, dev = tc._cuda_getCurrentRawStream, tc._cuda_getDevice
            _RAW_STREAM = lambda: get(dev())
        else:
            cur = _torch().cuda.current_stream
            _RAW_STREAM = lambda: cur().cuda_stream
    return C.c_void_p(_RAW_STREAM())


_DEVICES = None


def _here(*tensors):
    """Refuses operands of another GPU than the current one, where the library
    launches.  (Nothing to ask where there is one GPU: a microsecond a call.)"""
    global _DEVICES
    if _DEVICES is None:
        _DEVICES = _torch().cuda.device_count()
    if _DEVICES <= 1:
        return
    here = _torch().cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError(f"operands must be on the current device, cuda:{here}, not on "
                             f"cuda:{t.get_device()}")


def _on(stream):
    """New outputs within come from the pool of the stream that a call names, as
    those of any operation on it do.  (From the current stream's pool they
    could be memory that work pending there still uses.)"""
    if stream is None:
        return contextlib.nullcontext()
    cuda = _torch().cuda
    return cuda.stream(stream if isinstance(stream, cuda.Stream) else
                       cuda.ExternalStream(stream.cuda_stream))


def workspace(device=None):
    """A zeroed workspace tensor for the kernels' error word."""
    torch = _torch()
    return torch.zeros(workspace_bytes(), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


def _workspace_args(workspace):
    """Address and bytes of a workspace, which the kernels write: every byte it
    counts has to be its own, and on the GPU."""
    if workspace is None:
        return None, 0
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _here(workspace)
    return workspace.data_ptr(), workspace.nbytes


def _cfg_ptr(cfg):
    return C.byref(cfg) if cfg is not None else None


def _check_operand(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")


def _gemm_desc(a, b, out, batched: bool) -> _abi.GemmDesc:
    sa, sb, sc = a.stride(), b.stride(), out.stride()
    if not (a.is_cuda and b.is_cuda and out.is_cuda) or sa[-1] != 1 or sb[-1] != 1 or sc[-1] != 1:
        for t, nm in ((a, "a"), (b, "b"), (out, "out")):
            _check_operand(t, nm)
    ha, hb, hc = a.shape, b.shape, out.shape
    m, k, n = ha[-2], ha[-1], hb[-1]
    if hb[-2] != k or hc[-2] != m or hc[-1] != n:
        raise ValueError(f"shape mismatch: {tuple(ha)} x {tuple(hb)} -> {tuple(hc)}")
    _here(a, b, out)
    d = _abi.GemmDesc()
    d.m, d.n, d.k = m, n, k
    d.batch = ha[0] if batched else 1
    d.a, d.b, d.c = a.data_ptr(), b.data_ptr(), out.data_ptr()
    d.lda, d.ldb, d.ldc = sa[-2], sb[-2], sc[-2]
    if batched:
        if hb[0] != d.batch or hc[0] != d.batch:
            raise ValueError("batch sizes differ")
        d.stride_a, d.stride_b, d.stride_c = sa[0], sb[0], sc[0]
    d.a_dtype, d.b_dtype, d.c_dtype = _dtype_code(a), _dtype_code(b), _dtype_code(out)
    return d


def _alloc_out(shape, like, out_dtype, stream):
    torch = _torch()
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
          None: like.dtype}[out_dtype] if not isinstance(out_dtype, torch.dtype) else out_dtype
    with _on(stream):
        return torch.empty(shape, dtype=dt, device=like.device)


def gemm(a, b, out=None, out_dtype=None, cfg=None, workspace=None, stream=None):
    """out = a @ b for 2-D row-major CUDA tensors (fp16/bf16 in)."""
    if out is None:
        out = _alloc_out((a.shape[0], b.shape[1]), a, out_dtype, stream)
    d = _gemm_desc(a, b, out, batched=False)
    ws, wsb = _workspace_args(workspace)
    _check(load().tiles_gemm(C.byref(d), _cfg_ptr(cfg), ws, wsb, _stream_handle(stream)),
           "tiles_gemm")
    return out


def gemm_autotune(a, b, out, top_k=4, reps=5, workspace=None, stream=None, batched=None):
    """Time the planner's top_k configurations for out = a @ b (each with
    every last-round schedule it admits) and record the fastest as the tuned
    configuration of the problem, which later calls with cfg=None use.
    Overwrites `out`.  Returns (best Config, list of per-candidate dicts)."""
    if batched is None:
        batched = a.dim() == 3
    d = _gemm_desc(a, b, out, batched=batched)
    ws, wsb = _workspace_args(workspace)
    cap = 3 * top_k
    res = (_abi.TuneResult * cap)()
    n = C.c_int(0)
    best = _abi.Config()
    _check(load().tiles_gemm_autotune(C.byref(d), top_k, reps, ws, wsb, _stream_handle(stream),
                                      res, cap, C.byref(n), C.byref(best)),
           "tiles_gemm_autotune")
    rows = []
    for r in res[:min(n.value, cap)]:
        rows.append({"bm": r.cfg.bm, "bn": r.cfg.bn, "stages": r.cfg.stages,
                     "cta_group": r.cfg.cta_group, "tail_asked": r.cfg.tail,
                     "tail_mode": ["none", "n_halves", "k_split"][r.tail_mode],
                     "ksplit": r.ksplit, "status": r.status, "us": r.us})
    return best, rows


def tuned_lookup(sm_count, b, m, n, k, in_dtype, out_dtype):
    """The tuned Config of a problem (dtypes as "f16"/"bf16"/"f32" or codes),
    or None."""
    in_dtype = _abi.DTYPE_CODES.get(in_dtype, in_dtype)
    out_dtype = _abi.DTYPE_CODES.get(out_dtype, out_dtype)
    cfg = _abi.Config()
    s = load().tiles_tuned_lookup(sm_count, b, m, n, k, in_dtype, out_dtype, C.byref(cfg))
    if s == _abi.ERR_INFEASIBLE:
        return None
    _check(s, "tiles_tuned_lookup")
    return cfg


def tuned_save(path):
    _check(load().tiles_tuned_save(os.fsencode(path)), "tiles_tuned_save")


def tuned_load(path):
    _check(load().tiles_tuned_load(os.fsencode(path)), "tiles_tuned_load")


def tuned_clear():
    _check(load().tiles_tuned_clear(), "tiles_tuned_clear")


def gemm_batched(a, b, out=None, out_dtype=None, cfg=None, workspace=None, stream=None):
    """out[t] = a[t] @ b[t] for 3-D CUDA tensors."""
    if out is None:
        out = _alloc_out((a.shape[0], a.shape[1], b.shape[2]), a, out_dtype, stream)
    d = _gemm_desc(a, b, out, batched=True)
    ws, wsb = _workspace_args(workspace)
    _check(load().tiles_gemm_batched(C.byref(d), _cfg_ptr(cfg), ws, wsb, _stream_handle(stream)),
           "tiles_gemm_batched")
    return out


def _mirror(host, dev, nm):
    """A host tensor that mirrors a device tensor (same shape, dtype, strides)."""
    if host.is_cuda or tuple(host.shape) != tuple(dev.shape) or host.dtype != dev.dtype \
            or host.stride() != dev.stride():
        raise ValueError(f"{nm}: the host tensor must mirror its device tensor "
                         "(same shape, dtype and strides, in host memory)")


def gemm_host(a_host, b_host, out_host, a_dev, b_dev, out_dev, cfg=None, workspace=None,
              stream=None, chunks=4):
    """out_host = a_host @ b_host (2-D, or 3-D batched) through the device
    buffers a_dev, b_dev, out_dev: uploads, GEMMs and downloads in `chunks`
    overlapping pieces (tiles_gemm_host).  Host tensors should be pinned."""
    for h, dv, nm in ((a_host, a_dev, "a"), (b_host, b_dev, "b"), (out_host, out_dev, "out")):
        _mirror(h, dv, nm)
    d = _gemm_desc(*_batched3(a_dev, b_dev, out_dev), batched=True)
    ws, wsb = _workspace_args(workspace)
    _check(load().tiles_gemm_host(C.byref(d), _cfg_ptr(cfg), a_host.data_ptr(), b_host.data_ptr(),
                                  out_host.data_ptr(), chunks, ws, wsb, _stream_handle(stream)),
           "tiles_gemm_host")
    return out_host


def conv2d_host(x_host, w_host, y_host, x_dev, w_dev, y_dev, stride=(1, 1), pad=(0, 0),
                dil=(1, 1), tile_oh=16, cfg=None, workspace=None, stream=None, layout="nchw",
                chunks=4):
    """y_host = conv2d(x_host, w_host) through the device buffers x_dev, w_dev,
    y_dev: uploads, convolutions and downloads in `chunks` overlapping runs
    of images (tiles_conv2d_host).  Host tensors should be pinned."""
    for h, dv, nm in ((x_host, x_dev, "x"), (w_host, w_dev, "w"), (y_host, y_dev, "y")):
        _mirror(h, dv, nm)
    d = _conv_desc(x_dev, w_dev, stride, pad, dil, y_dev, layout)
    ws, wsb = _workspace_args(workspace)
    _check(load().tiles_conv2d_host(C.byref(d), tile_oh, _cfg_ptr(cfg), x_host.data_ptr(),
                                    w_host.data_ptr(), y_host.data_ptr(), chunks, ws, wsb,
                                    _stream_handle(stream)),
           "tiles_conv2d_host")
    return y_host


_OUT_HW = {}


def conv_out_hw(h, w, kh, kw, stride, pad, dil):
    """Output height and width of a convolution (tiles_conv_out_hw; the
    library's answer is kept per geometry, so repeated calls skip it)."""
    key = (h, w, kh, kw, tuple(stride), tuple(pad), tuple(dil))
    hit = _OUT_HW.get(key)
    if hit is not None:
        return hit
    d = _abi.ConvDesc()
    d.n, d.c, d.h, d.w, d.c_out, d.kh, d.kw = 1, 1, h, w, 1, kh, kw
    d.sh, d.sw = stride
    d.ph, d.pw = pad
    d.dh, d.dw = dil
    oh, ow = C.c_int32(0), C.c_int32(0)
    _check(load().tiles_conv_out_hw(C.byref(d), C.byref(oh), C.byref(ow)), "tiles_conv_out_hw")
    if len(_OUT_HW) < 4096:
        _OUT_HW[key] = (oh.value, ow.value)
    return oh.value, ow.value


def _conv_desc(x, w, stride, pad, dil, out, layout):
    for t, nm in ((x, "x"), (w, "w")):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{nm} must be a contiguous CUDA tensor")
    _here(x, w)
    if layout == "nchw":
        n, c, h, wd = x.shape
    elif layout == "nhwc":
        n, h, wd, c = x.shape
    else:
        raise ValueError(f"unknown layout {layout!r}")
    co, c2, kh, kw = w.shape
    if c2 != c:
        raise ValueError("channel mismatch")
    d = _abi.ConvDesc()
    d.n, d.c, d.h, d.w = n, c, h, wd
    d.c_out, d.kh, d.kw = co, kh, kw
    d.sh, d.sw = stride
    d.ph, d.pw = pad
    d.dh, d.dw = dil
    d.in_dtype = _dtype_code(x)
    if _dtype_code(w) != d.in_dtype:
        raise TypeError("x and w must share a dtype")
    d.x_layout = _abi.LAYOUT_NHWC if layout == "nhwc" else _abi.LAYOUT_NCHW
    d.x, d.wt = x.data_ptr(), w.data_ptr()
    if out is not None:
        if not out.is_cuda or not out.is_contiguous():
            raise ValueError("out must be a contiguous CUDA tensor")
        _here(out)
        d.y = out.data_ptr()
        d.out_dtype = _dtype_code(out)
    return d


def conv_out_shape(x, w, stride=(1, 1), pad=(0, 0), dil=(1, 1), layout="nchw"):
    n, c, h, wd = x.shape if layout == "nchw" else (x.shape[0], x.shape[3], x.shape[1], x.shape[2])
    co, _, kh, kw = w.shape
    oh, ow = conv_out_hw(h, wd, kh, kw, stride, pad, dil)
    return (n, co, oh, ow)


def conv_workspace(x, w, stride=(1, 1), pad=(0, 0), dil=(1, 1), tile_oh=16, layout="nchw"):
    """A zeroed workspace for the TMA im2col producer of this convolution."""
    torch = _torch()
    d = _conv_desc(x, w, stride, pad, dil, None, layout)
    nbytes = int(load().tiles_conv_workspace_bytes(C.byref(d), tile_oh))
    if nbytes == 0:
        raise ValueError("invalid convolution arguments")
    return torch.zeros(nbytes, dtype=torch.uint8, device=x.device)


def conv2d_htiled(x, w, stride=(1, 1), pad=(0, 0), dil=(1, 1), tile_oh=16, out=None,
                  out_dtype=None, cfg=None, workspace=None, stream=None, layout="nchw"):
    """conv2d with OIHW weights and NCHW output, as an implicit GEMM per output
    H-tile; x is NCHW or NHWC (layout).  With a workspace of conv_workspace
    size the im2col operand is built by TMA, else gathered by threads."""
    shape = conv_out_shape(x, w, stride, pad, dil, layout)
    if out is None:
        out = _alloc_out(shape, x, out_dtype, stream)
    if not out.is_contiguous() or tuple(out.shape) != shape:
        raise ValueError("out must be contiguous with shape (n, c_out, oh, ow)")
    d = _conv_desc(x, w, stride, pad, dil, out, layout)
    ws, wsb = _workspace_args(workspace)
    _check(load().tiles_conv2d_htiled(C.byref(d), tile_oh, _cfg_ptr(cfg), ws, wsb,
                                      _stream_handle(stream)), "tiles_conv2d_htiled")
    return out


def conv2d_tiled(x, w, stride=(1, 1), pad=(0, 0), dil=(1, 1), tile_oh=16, tile_ow=0, tile_n=0,
                 out=None, out_dtype=None, cfg=None, workspace=None, stream=None, layout="nchw"):
    """conv2d tiled over the batch (tile_n images, no halo), the output
    height (tile_oh rows) and the output width (tile_ow columns, the same
    slicing formulas as the rows); 0 means the whole batch or width."""
    shape = conv_out_shape(x, w, stride, pad, dil, layout)
    if out is None:
        out = _alloc_out(shape, x, out_dtype, stream)
    if not out.is_contiguous() or tuple(out.shape) != shape:
        raise ValueError("out must be contiguous with shape (n, c_out, oh, ow)")
    d = _conv_desc(x, w, stride, pad, dil, out, layout)
    ws, wsb = _workspace_args(workspace)
    _check(load().tiles_conv2d_tiled(C.byref(d), tile_oh, tile_ow, tile_n, _cfg_ptr(cfg), ws,
                                     wsb, _stream_handle(stream)), "tiles_conv2d_tiled")
    return out


def _batched3(a, b, out):
    if a.dim() == 2:
        return a.unsqueeze(0), b.unsqueeze(0), out.unsqueeze(0)
    return a, b, out


def gemm_schedule(a, b, out, cfg=None, workspace=None):
    """The launch geometry a GEMM call with this workspace would use (2-D
    tensors count as a batch of one)."""
    d = _gemm_desc(*_batched3(a, b, out), batched=True)
    sch = _abi.Schedule()
    _, wsb = _workspace_args(workspace)
    _check(load().tiles_gemm_schedule(C.byref(d), _cfg_ptr(cfg), wsb, C.byref(sch)),
           "tiles_gemm_schedule")
    return sch


def gemm_workspace(a, b, out, cfg=None):
    """A zeroed workspace large enough for this GEMM's schedule under cfg (the
    partial tiles of a K-split last round, when that is the schedule)."""
    torch = _torch()
    d = _gemm_desc(*_batched3(a, b, out), batched=True)
    n = int(load().tiles_gemm_workspace_bytes(C.byref(d), _cfg_ptr(cfg)))
    if n == 0:
        # The call returns 0 on invalid arguments; tiles_last_error says why.
        raise TilesError(_abi.ERR_INVALID_ARG, "tiles_gemm_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=a.device)


def gemm_noalloc(a, b, out=None, out_dtype=None, cfg=None, stream=None, wait=False):
    """out[t] = a[t] @ b[t] (3-D tensors) without a workspace: for callers
    that cannot allocate device memory.  The library's static scratch takes
    the workspace's place; wait=True synchronises and reports a timeout."""
    if out is None:
        out = _alloc_out((a.shape[0], a.shape[1], b.shape[2]), a, out_dtype, stream)
    d = _gemm_desc(a, b, out, batched=True)
    _check(load().tiles_gemm_noalloc(C.byref(d), _cfg_ptr(cfg), _stream_handle(stream),
                                     1 if wait else 0), "tiles_gemm_noalloc")
    return out


def check(workspace=None, stream=None) -> None:
    """Synchronise and raise TilesError if a kernel's bounded wait expired."""
    ws, _ = _workspace_args(workspace)
    _check(load().tiles_check(ws, _stream_handle(stream)), "tiles_check")


def selftest_wait_timeout(workspace, limit_ns: int, stream=None) -> None:
    _check(load().tiles_selftest_wait_timeout(_workspace_args(workspace)[0], limit_ns,
                                              _stream_handle(stream)),
           "tiles_selftest_wait_timeout")


def selftest_drop_stage(stage: int, limit_ns: int) -> None:
    """Arm a planted fault for this thread's next GEMM or TMA convolution
    launch (tiles_selftest_drop_stage); stage < 0 disarms."""
    _check(load().tiles_selftest_drop_stage(stage, limit_ns), "tiles_selftest_drop_stage")


# ---- norms, 8-bit products and products grouped by expert ------------------------
#
# These calls are short: a decoding step's norm or product takes a few
# microseconds on the GPU, less than a dozen Python calls take.  So each one
# goes through the compiled module first (_calls: checks, allocation and launch
# without Python objects in between), which returns None for what it does not
# take.  The Python function then makes the same call the long way, where
# _refuse finds what is wrong with the arguments.
#
# A call runs on `stream`, or on the current stream.  Its new outputs belong to
# that stream, as after any PyTorch operation on it: used on another one, they
# are the caller's to order (wait_stream, record_stream).  Outputs that the
# caller gives may not overlap an input, but for a norm's h_out.


class _NoCalls:
    """Stands in for the compiled calls where they were not built or do not load."""

    rmsnorm = rmsnorm_grad = product_fp8 = grouped_gemm = grouped_wgrad = \
        staticmethod(lambda *args: None)


_CALLS = None


def _compiled():
    global _CALLS
    _torch()
    lib = load()
    calls = _NoCalls
    if os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_calls.so")):
        try:
            from . import _calls as calls
        except ImportError as e:
            # Of another PyTorch, say: the long way does the same.
            warnings.warn(f"the compiled calls do not load, build them again: {e}")
        else:
            calls.bind(*(C.cast(getattr(lib, "tiles_" + name), C.c_void_p).value for name in
                         ("rmsnorm", "rmsnorm_grad", "gemm_fp8", "grouped_gemm", "grouped_wgrad")))
    _CALLS = calls
    return _CALLS


SCALE_BLOCK = 128     # columns (and weight rows) that share one scale

# The descriptors of include/tiles.h, field by field (_abi has their names).
_NORM = struct.Struct("2q6Q6qf3i")
_NORM_GRAD = struct.Struct("2q6Q4qf3i")
_PRODUCT = struct.Struct("4q6Q9q4i")
_WGRAD = struct.Struct("4q4Q4q2i")


def _codes():
    """Codes of the floating types, by torch dtype."""
    _torch()
    if _DTYPE_CODES is None:
        _dtype_code(_torch().empty(0))
    return _DTYPE_CODES


def _raw_stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _RAW_STREAM is None:
        _stream_handle(None)
    return _RAW_STREAM()


def _blocks(n):
    return (n + SCALE_BLOCK - 1) // SCALE_BLOCK


def _refuse(*rules):
    """Raises for the first (name, tensor, shape, dtype) that is not a CUDA tensor
    of that shape and type with unit stride in its last dimension (shape:
    any where None; dtype: a type or several)."""
    for name, t, shape, dtype in rules:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must have unit stride in its last dimension")
        kinds = dtype if isinstance(dtype, (tuple, set)) else (dtype,)
        if t.dtype not in kinds:
            raise TypeError(f"{name} must be {' or '.join(sorted(map(str, kinds)))}, not {t.dtype}")
    raise ValueError("unsupported arguments")


def _matrix(t, name):
    """Shape and strides of a matrix; the pitch of a single row, which nothing
    uses, as whole 16-byte pieces."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a matrix")
    rows, cols = shape
    ld, unit = t.stride()
    return rows, cols, (ld if rows > 1 else (cols + 15) // 16 * 16), (1 if cols <= 1 else unit)


def _rmsnorm(x, weight, residual, eps, out, scales, h_out, stream, fp8):
    torch = _TORCH or _torch()
    codes = _DTYPE_CODES or _codes()
    rows, cols, ldx, unit = _matrix(x, "x")
    shape, dtype, device = x.shape, x.dtype, x.device
    code, wcode = codes.get(dtype), codes.get(weight.dtype)
    given = out is not None
    if given:
        _, _, ldy, uy = _matrix(out, "out")
    elif fp8:
        ldy = (cols + 15) // 16 * 16          # whole 16-byte pieces, as the products need
        out = torch.empty((rows, ldy), dtype=torch.float8_e4m3fn, device=device)
        if ldy != cols:
            out = out[:, :cols]
    else:
        out, ldy = torch.empty(shape, dtype=dtype, device=device), cols
    ps = sr = sb = 0
    if fp8:
        nb = (cols + 127) // 128
        if scales is None:
            sr, sb = 1, rows or 1             # stored block by block: the products' fastest order
            scales = torch.empty_strided((rows, nb), (sr, sb), dtype=torch.float32, device=device)
        else:
            if scales.shape != (rows, nb) or scales.dtype != torch.float32 or not scales.is_cuda:
                raise ValueError(f"scales must be a float32 CUDA tensor of shape {(rows, nb)}")
            sr, sb = scales.stride()
        ps = scales.data_ptr()
    h, pr, ldr, ph, ldh, ok = x, 0, 0, 0, 0, True
    if residual is not None:
        _, _, ldr, ur = _matrix(residual, "residual")
        ok = ur == 1 and residual.shape == shape and residual.dtype == dtype and residual.is_cuda
        pr = residual.data_ptr()
        if h_out is None:
            h, ldh = torch.empty(shape, dtype=dtype, device=device), cols
            ph = h.data_ptr()
    if h_out is not None:
        h = h_out
        _, _, ldh, uh = _matrix(h, "h_out")
        ok = ok and uh == 1 and h.shape == shape and h.dtype == dtype and h.is_cuda
        ph = h.data_ptr()
    if given:
        ok = ok and uy == 1 and out.shape == shape and out.is_cuda and \
            out.dtype == (torch.float8_e4m3fn if fp8 else dtype)
    if not (ok and unit == 1 and x.is_cuda and weight.is_cuda and code is not None and
            wcode is not None and weight.shape == (cols,) and (cols == 1 or weight.stride(0) == 1)):
        _refuse(("x", x, None, set(codes)), ("weight", weight, (cols,), set(codes)),
                ("residual", residual, shape, dtype),
                ("h_out", h_out, shape, dtype),
                ("out", out if given else None, shape, torch.float8_e4m3fn if fp8 else dtype))
    _here(x, weight, residual, out, scales, h)
    d = _NORM.pack(rows, cols, x.data_ptr(), pr, weight.data_ptr(), ph, out.data_ptr(), ps, ldx, ldr,
                   ldh, ldy, sr, sb, eps, code, wcode, _abi.E4M3 if fp8 else code)
    _check(load().tiles_rmsnorm(d, _raw_stream(stream)), "tiles_rmsnorm")
    return out, scales, h


def rmsnorm(x, weight, residual=None, eps=1e-6, out=None, h_out=None, stream=None):
    """h = x + residual and y = h * (mean(h^2) + eps)^(-1/2) * weight, row by
    row of a matrix; returns (y, h) in x's type.  Without a residual h is x
    itself, or a copy of it in h_out.  h_out may be the residual (updated in
    place)."""
    r = (_CALLS or _compiled()).rmsnorm(x, weight, residual, eps, out, None, h_out, stream, False)
    if r is None:
        with _on(stream):
            r = _rmsnorm(x, weight, residual, eps, out, None, h_out, stream, False)
    return r[0], r[2]


def rmsnorm_fp8(x, weight, residual=None, eps=1e-6, out=None, scales=None, h_out=None,
                stream=None):
    """The norm of rmsnorm with y in 8 bits: returns (q, scales, h), e4m3
    values and one fp32 scale per row and 128 columns, y ~ q * scale.  New
    scales are stored block by block (a transposed view, rows x blocks),
    which the products read fastest."""
    r = (_CALLS or _compiled()).rmsnorm(x, weight, residual, eps, out, scales, h_out, stream, True)
    if r is None:
        with _on(stream):
            r = _rmsnorm(x, weight, residual, eps, out, scales, h_out, stream, True)
    return r


def rmsnorm_grad_workspace(x):
    """A zeroed workspace for rmsnorm_grad on matrices of x's shape."""
    torch = _torch()
    rows, cols = x.shape
    n = int(load().tiles_rmsnorm_grad_workspace_bytes(rows, cols))
    if n == 0:
        raise TilesError(_abi.ERR_INVALID_ARG, "tiles_rmsnorm_grad_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=x.device)


def rmsnorm_grad(dy, h, weight, eps=1e-6, dh=None, dx_out=None, dweight_out=None, workspace=None,
                 stream=None):
    """Gradients of rmsnorm at h, given those of y (dy) and, where h is used
    past the norm, of h (dh): returns (dx, dweight).  dx, in h's type, is the
    gradient of x and of the residual alike; dweight is fp32."""
    r = (_CALLS or _compiled()).rmsnorm_grad(dy, h, weight, eps, dh, dx_out, dweight_out,
                                             workspace, stream)
    if r is not None:
        return r
    torch = _TORCH or _torch()
    codes = _DTYPE_CODES or _codes()
    rows, cols, ldh, unit = _matrix(h, "h")
    shape, dtype = h.shape, h.dtype
    code, wcode = codes.get(dtype), codes.get(weight.dtype)
    _, _, lddy, ud = _matrix(dy, "dy")
    lddh = pdh = 0
    ok = True
    if dh is not None:
        _, _, lddh, u = _matrix(dh, "dh")
        ok = u == 1 and dh.shape == shape and dh.dtype == dtype and dh.is_cuda
        pdh = dh.data_ptr()
    dx, dw = dx_out, dweight_out
    if dx is None:
        with _on(stream):
            dx, lddx = torch.empty(shape, dtype=dtype, device=h.device), cols
    else:
        _, _, lddx, u = _matrix(dx, "dx_out")
        ok = ok and u == 1 and dx.shape == shape and dx.dtype == dtype and dx.is_cuda
    if dw is None:
        with _on(stream):
            dw = torch.empty(cols, dtype=torch.float32, device=h.device)
    else:
        ok = ok and dw.shape == (cols,) and dw.dtype == torch.float32 and dw.is_cuda and \
            (cols == 1 or dw.stride(0) == 1)
    if not (ok and unit == 1 and ud == 1 and h.is_cuda and dy.is_cuda and weight.is_cuda and
            code is not None and wcode is not None and dy.shape == shape and dy.dtype == dtype and
            weight.shape == (cols,) and (cols == 1 or weight.stride(0) == 1)):
        _refuse(("h", h, None, set(codes)), ("dy", dy, shape, dtype),
                ("weight", weight, (cols,), set(codes)), ("dh", dh, shape, dtype),
                ("dx_out", dx_out, shape, dtype),
                ("dweight_out", dweight_out, (cols,), torch.float32))
    _here(dy, h, weight, dh, dx, dw)
    d = _NORM_GRAD.pack(rows, cols, dy.data_ptr(), h.data_ptr(), weight.data_ptr(), pdh,
                        dx.data_ptr(), dw.data_ptr(), lddy, ldh, lddh, lddx, eps, code, wcode, 0)
    ws, wsb = _workspace_args(workspace)
    _check(load().tiles_rmsnorm_grad(d, ws, wsb, _raw_stream(stream)), "tiles_rmsnorm_grad")
    return dx, dw


def quantize_fp8(x, block_rows=1, stream=None):
    """e4m3 values and fp32 scales of x (a matrix, or a batch of them): one
    scale per row and 128 columns (block_rows 1: activations; the scales are
    stored block by block, as a view rows x blocks) or per 128 x 128
    (block_rows 128: weights)."""
    torch = _torch()
    if not x.is_cuda or x.dim() not in (2, 3):
        raise ValueError("x must be a CUDA matrix or a batch of them")
    if x.shape[-1] > 1 and x.stride(-1) != 1:
        raise ValueError("x must have unit stride in its last dimension")
    if block_rows not in (1, SCALE_BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    *lead, rows, cols = x.shape
    batch = lead[0] if lead else 1
    pitch = (cols + 15) // 16 * 16
    nb = _blocks(cols)
    with _on(stream):
        q = torch.empty((*lead, rows, pitch), dtype=torch.float8_e4m3fn, device=x.device)[..., :cols]
        if block_rows == 1:
            scales = torch.empty((*lead, nb, rows), dtype=torch.float32,
                                 device=x.device).transpose(-1, -2)
        else:
            scales = torch.empty((*lead, _blocks(rows), nb), dtype=torch.float32, device=x.device)
    _here(x)
    d = _abi.QuantizeDesc(batch, rows, cols, x.data_ptr(), q.data_ptr(), scales.data_ptr(),
                          x.stride(-2) if rows > 1 else max(x.stride(-2), cols),
                          x.stride(0) if lead else 0, pitch, q.stride(0) if lead else 0,
                          scales.stride(-2), scales.stride(-1), scales.stride(0) if lead else 0,
                          _dtype_code(x), block_rows)
    _check(load().tiles_quantize_fp8(C.byref(d), _stream_handle(stream)), "tiles_quantize_fp8")
    return q, scales


def _weight(b, grouped, name):
    """Shape (..., rows, cols), row pitch, group stride and unit stride of a weight."""
    shape, st = b.shape, b.stride()
    if len(shape) != (3 if grouped else 2):
        raise ValueError(f"{name} must have {3 if grouped else 2} dimensions")
    cols = shape[-1]
    ld = st[-2] if shape[-2] > 1 else (cols + 15) // 16 * 16
    return shape, ld, (st[0] if grouped else 0), (1 if cols <= 1 else st[-1])


def _product_fp8(a, a_scales, b, b_scales, offsets, out, out_dtype, workspace, stream, where):
    torch = _TORCH or _torch()
    codes = _DTYPE_CODES or _codes()
    grouped = offsets is not None
    m, k, lda, ua = _matrix(a, "a")
    bshape, ldb, stride_b, ub = _weight(b, grouped, "b")
    n = bshape[-2]
    kb, nb = (k + 127) // 128, (n + 127) // 128
    sbs = b_scales.stride()
    if grouped:
        groups = bshape[0]
        scales_shape, sbg, off = (groups, nb, kb), sbs[0], offsets.data_ptr()
        ok = offsets.shape == (groups + 1,) and offsets.dtype == torch.int32 and \
            offsets.is_cuda and offsets.stride(0) == 1
    else:
        groups = sbg = off = 0
        scales_shape, ok = (nb, kb), True
    given = out is not None
    if given:
        _, _, ldc, u = _matrix(out, "out")
        ok = ok and u == 1 and out.shape == (m, n) and out.is_cuda and out.dtype in codes
    else:
        dt = out_dtype if isinstance(out_dtype, torch.dtype) else \
            _TYPES(torch)["bf16" if out_dtype is None else out_dtype]
        out, ldc = torch.empty((m, n), dtype=dt, device=a.device), n
    fp8 = torch.float8_e4m3fn
    if not (ok and ua == 1 and ub == 1 and a.dtype == fp8 and b.dtype == fp8 and a.is_cuda and
            b.is_cuda and bshape[-1] == k and a_scales.shape == (m, kb) and
            b_scales.shape == scales_shape and a_scales.dtype == torch.float32 and
            b_scales.dtype == torch.float32 and a_scales.is_cuda and b_scales.is_cuda):
        for s, shape, name in ((a_scales, (m, kb), "a_scales"), (b_scales, scales_shape, "b_scales")):
            if s.shape != shape or s.dtype != torch.float32 or not s.is_cuda:
                raise ValueError(f"{name} must be a float32 CUDA tensor of shape {shape}")
        _refuse(("a", a, None, fp8), ("b", b, (*bshape[:-1], k), fp8),
                ("offsets", offsets, (groups + 1,), torch.int32),
                ("out", out if given else None, (m, n), set(codes)))
    _here(a, a_scales, b, b_scales, offsets, out)
    sar, sab = a_scales.stride()
    d = _PRODUCT.pack(m, n, k, groups, off, a.data_ptr(), b.data_ptr(), out.data_ptr(),
                      a_scales.data_ptr(), b_scales.data_ptr(), lda, ldb, ldc, stride_b, sar, sab,
                      sbs[-2], sbs[-1], sbg, _abi.E4M3, codes[out.dtype], _abi.B_NK, 0)
    ws, wsb = _workspace_args(workspace)
    fn = load().tiles_grouped_gemm if grouped else load().tiles_gemm_fp8
    _check(fn(d, ws, wsb, _raw_stream(stream)), where)
    return out


_TYPE_NAMES = None


def _TYPES(torch):
    """Types by the names that out_dtype takes."""
    global _TYPE_NAMES
    if _TYPE_NAMES is None:
        _TYPE_NAMES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
    return _TYPE_NAMES


def gemm_fp8(a, a_scales, b, b_scales, out=None, out_dtype=None, workspace=None, stream=None):
    """out[i][j] = sum over blocks t of 128 of a_scales[i][t] * b_scales[j//128][t]
    * (a[i] . b[j] within t): e4m3 rows (m x k, as rmsnorm_fp8 and
    quantize_fp8 give them) times an e4m3 weight stored n x k.  out is bf16
    unless out_dtype ("f32", "f16", "bf16") says otherwise."""
    r = (_CALLS or _compiled()).product_fp8(a, a_scales, b, b_scales, None, out, out_dtype,
                                            workspace, stream)
    if r is None:
        with _on(stream):
            r = _product_fp8(a, a_scales, b, b_scales, None, out, out_dtype, workspace, stream,
                             "tiles_gemm_fp8")
    return r


def grouped_gemm_fp8(a, a_scales, b, b_scales, offsets, out=None, out_dtype=None, workspace=None,
                     stream=None):
    """gemm_fp8 with a weight per group (b: groups x n x k): rows offsets[g] ..
    offsets[g+1] - 1 of a meet b[g].  offsets is an int32 CUDA vector that
    only the kernel reads.  Rows outside every group are not written."""
    r = (_CALLS or _compiled()).product_fp8(a, a_scales, b, b_scales, offsets, out, out_dtype,
                                            workspace, stream)
    if r is None:
        with _on(stream):
            r = _product_fp8(a, a_scales, b, b_scales, offsets, out, out_dtype, workspace, stream,
                             "tiles_grouped_gemm")
    return r


def grouped_gemm(a, b, offsets, trans_b=False, out=None, out_dtype=None, workspace=None,
                 stream=None):
    """out[i] = a[i] @ b[g] for the rows i of group g, offsets[g] <= i <
    offsets[g+1]: fp16/bf16 rows (m x k) and weights (groups x k x n).  With
    trans_b the weights are groups x n x k and out[i] = a[i] @ b[g]^T, which
    is the gradient of the rows when a is that of the products.  offsets is
    an int32 CUDA vector that only the kernel reads.  Rows outside every
    group are not written."""
    r = (_CALLS or _compiled()).grouped_gemm(a, b, offsets, trans_b, out, out_dtype, workspace,
                                             stream)
    if r is not None:
        return r
    torch = _TORCH or _torch()
    codes = _DTYPE_CODES or _codes()
    m, k, lda, ua = _matrix(a, "a")
    bshape, ldb, stride_b, ub = _weight(b, True, "b")
    groups, bk, n = (bshape[0], bshape[2], bshape[1]) if trans_b else bshape
    dtype = a.dtype
    given, ok = out is not None, True
    if given:
        _, _, ldc, u = _matrix(out, "out")
        ok = u == 1 and out.shape == (m, n) and out.is_cuda and out.dtype in codes
    else:
        dt = dtype if out_dtype is None else \
            out_dtype if isinstance(out_dtype, torch.dtype) else _TYPES(torch)[out_dtype]
        with _on(stream):
            out, ldc = torch.empty((m, n), dtype=dt, device=a.device), n
    if not (ok and ua == 1 and ub == 1 and bk == k and b.dtype == dtype and dtype in codes and
            a.is_cuda and b.is_cuda and offsets.shape == (groups + 1,) and offsets.is_cuda and
            offsets.dtype == torch.int32 and offsets.stride(0) == 1):
        if offsets.dtype != torch.int32:
            raise ValueError("offsets must be int32")
        _refuse(("a", a, None, set(codes)),
                ("b", b, (groups, n, k) if trans_b else (groups, k, n), dtype),
                ("offsets", offsets, (groups + 1,), torch.int32),
                ("out", out if given else None, (m, n), set(codes)))
    _here(a, b, offsets, out)
    d = _PRODUCT.pack(m, n, k, groups, offsets.data_ptr(), a.data_ptr(), b.data_ptr(),
                      out.data_ptr(), 0, 0, lda, ldb, ldc, stride_b, 0, 0, 0, 0, 0, codes[dtype],
                      codes[out.dtype], _abi.B_NK if trans_b else _abi.B_KN, 0)
    ws, wsb = _workspace_args(workspace)
    _check(load().tiles_grouped_gemm(d, ws, wsb, _raw_stream(stream)), "tiles_grouped_gemm")
    return out


def grouped_wgrad(a, dc, offsets, out=None, out_dtype=None, workspace=None, stream=None):
    """out[g] = a_g^T @ dc_g over the rows of group g: the weight gradients
    (groups x k x n) of out = grouped_gemm(a, w, offsets), given dc.  An
    empty group's gradient is zero."""
    r = (_CALLS or _compiled()).grouped_wgrad(a, dc, offsets, out, out_dtype, workspace, stream)
    if r is not None:
        return r
    torch = _TORCH or _torch()
    codes = _DTYPE_CODES or _codes()
    m, k, lda, ua = _matrix(a, "a")
    md, n, lddc, ud = _matrix(dc, "dc")
    dtype = a.dtype
    groups = offsets.shape[0] - 1
    given, ok = out is not None, True
    if given:
        oshape, ldw, stride_dw, u = _weight(out, True, "out")
        ok = u == 1 and oshape == (groups, k, n) and out.is_cuda and out.dtype in codes
    else:
        dt = dtype if out_dtype is None else \
            out_dtype if isinstance(out_dtype, torch.dtype) else _TYPES(torch)[out_dtype]
        with _on(stream):
            out = torch.empty((groups, k, n), dtype=dt, device=a.device)
        ldw, stride_dw = n, k * n
    if not (ok and ua == 1 and ud == 1 and md == m and dc.dtype == dtype and dtype in codes and
            a.is_cuda and dc.is_cuda and offsets.is_cuda and offsets.dtype == torch.int32 and
            offsets.dim() == 1 and offsets.stride(0) == 1):
        _refuse(("a", a, None, set(codes)), ("dc", dc, (m, n), dtype),
                ("offsets", offsets, (groups + 1,), torch.int32),
                ("out", out if given else None, (groups, k, n), set(codes)))
    _here(a, dc, offsets, out)
    d = _WGRAD.pack(m, k, n, groups, offsets.data_ptr(), a.data_ptr(), dc.data_ptr(),
                    out.data_ptr(), lda, lddc, ldw, stride_dw, codes[dtype], codes[out.dtype])
    ws, wsb = _workspace_args(workspace)
    _check(load().tiles_grouped_wgrad(d, ws, wsb, _raw_stream(stream)), "tiles_grouped_wgrad")
    return out
