// The short calls on PyTorch tensors (norms, 8-bit and grouped products, routing,
// clipping), as a Python module.  A decoding step's norm or product takes a few microseconds
// on the GPU, and marshalling it in Python takes more: here the arguments are
// read, checked, the outputs allocated and the C call made without going
// through Python objects.  (Per call on the host: the norm of one row of 4096
// with residual and 8-bit output 4.7 us against 12.1 in Python, the 8-bit
// product of 16 rows 3.7 against 9.2; the C call is 2.0 to 2.6 of it.)
//
// Each function takes the arguments of its Python wrapper by position and
// returns None for anything it does not take or that fails: the wrapper then
// goes the long way, which names what is wrong.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <optional>
#include <vector>

#include "tiles.h"

namespace {

struct Refused {};

void require(bool ok) {
    if (!ok) throw Refused{};
}

// Addresses of the C calls, from the library that the package has loaded.
struct Calls {
    int (*rmsnorm)(const tiles_rmsnorm_desc*, void*);
    int (*rmsnorm_grad)(const tiles_rmsnorm_grad_desc*, void*, size_t, void*);
    int (*gemm_fp8)(const tiles_product_desc*, void*, size_t, void*);
    int (*grouped_gemm)(const tiles_product_desc*, void*, size_t, void*);
    int (*grouped_wgrad)(const tiles_wgrad_desc*, void*, size_t, void*);
    int (*layernorm)(const tiles_layernorm_desc*, void*);
    int (*layernorm_grad)(const tiles_layernorm_grad_desc*, void*, size_t, void*);
    size_t (*layernorm_grad_workspace_bytes)(int64_t, int64_t);
    int (*expert_sort)(const tiles_expert_sort_desc*, void*, size_t, void*);
    size_t (*expert_sort_workspace_bytes)(int64_t, int64_t, int64_t);
    int (*expert_dispatch)(const tiles_dispatch_desc*, void*);
    int (*expert_combine)(const tiles_combine_desc*, void*);
    int (*expert_combine_grad)(const tiles_combine_desc*, void*);
    int (*grad_norm)(const tiles_grad_tensor*, int64_t, float*, void*, size_t, void*);
    int (*clip_grads)(const tiles_grad_tensor*, int64_t, float, float, float*, void*, size_t, void*);
    size_t (*grad_norm_workspace_bytes)(int64_t);
} calls;

constexpr auto kE4m3 = at::ScalarType::Float8_e4m3fn;

int code_of(at::ScalarType t) {
    switch (t) {
        case at::ScalarType::Half: return TILES_F16;
        case at::ScalarType::BFloat16: return TILES_BF16;
        case at::ScalarType::Float: return TILES_F32;
        default: throw Refused{};
    }
}

bool several_devices() {
    static const bool yes = c10::cuda::device_count() > 1;
    return yes;
}

// Tensors are read where Python holds them: the arguments outlive the call.
// They are on the current device, where the library launches.
const at::Tensor* optional_tensor(PyObject* o) {
    if (o == Py_None) return nullptr;
    require(THPVariable_Check(o));
    const at::Tensor* t = &THPVariable_Unpack(o);
    require(t->is_cuda() && (!several_devices() || t->get_device() == c10::cuda::current_device()));
    return t;
}

const at::Tensor& tensor(PyObject* o) {
    const at::Tensor* t = optional_tensor(o);
    require(t != nullptr);
    return *t;
}

// Rows and columns of a matrix with unit column stride, and its row pitch (of
// a single row, which nothing uses, whole 16-byte pieces).
struct Matrix {
    int64_t rows, cols, ld;

    explicit Matrix(const at::Tensor& t) {
        require(t.dim() == 2);
        rows = t.size(0);
        cols = t.size(1);
        require(cols <= 1 || t.stride(1) == 1);
        ld = rows > 1 ? t.stride(0) : (cols + 15) / 16 * 16;
    }
    bool like(const Matrix& m) const { return rows == m.rows && cols == m.cols; }
};

// The same of a weight, with the stride between groups.
struct Weight {
    int64_t groups, rows, cols, ld, stride;

    Weight(const at::Tensor& t, bool grouped) {
        require(t.dim() == (grouped ? 3 : 2));
        const int d = grouped ? 1 : 0;
        groups = grouped ? t.size(0) : 0;
        rows = t.size(d);
        cols = t.size(d + 1);
        require(cols <= 1 || t.stride(d + 1) == 1);
        ld = rows > 1 ? t.stride(d) : (cols + 15) / 16 * 16;
        stride = grouped ? t.stride(0) : 0;
    }
};

bool is_vector(const at::Tensor& t, int64_t n, at::ScalarType dtype) {
    return t.dim() == 1 && t.size(0) == n && (n <= 1 || t.stride(0) == 1) &&
           t.scalar_type() == dtype;
}

at::Tensor empty(const at::Tensor& like, at::IntArrayRef size, at::IntArrayRef stride,
                 at::ScalarType dtype) {
    return at::Tensor(at::detail::empty_strided_cuda(size, stride, dtype, like.device()));
}

at::Tensor empty_matrix(const at::Tensor& like, int64_t rows, int64_t cols, int64_t ld,
                        at::ScalarType dtype) {
    return empty(like, {rows, cols}, {ld, 1}, dtype);
}

// The stream that a call names, or the current one.  While this lives it is
// the current one: new outputs come from its pool, as those of any operation on
// it do.  (From another stream's pool they could be memory that work pending
// there still uses.)
struct OnStream {
    void* at;
    std::optional<c10::cuda::CUDAStreamGuard> guard;

    explicit OnStream(PyObject* o) : at(c10::cuda::getCurrentCUDAStream().stream()) {
        if (o == Py_None) return;
        PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
        require(v != nullptr);
        void* s = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
        require(!PyErr_Occurred());
        if (s == at) return;
        at = s;
        guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s),
                                                       c10::cuda::current_device()));
    }
};

struct Workspace {
    void* at = nullptr;
    size_t bytes = 0;

    explicit Workspace(PyObject* o) {
        if (const at::Tensor* t = optional_tensor(o)) {
            require(t->is_contiguous());           // every byte it counts is its own
            at = t->data_ptr();
            bytes = t->nbytes();
        }
    }
};

float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    require(!PyErr_Occurred());
    return static_cast<float>(v);
}

// The type that out_dtype names ("f32", "f16", "bf16" or a torch type).
at::ScalarType out_type(PyObject* o, at::ScalarType otherwise) {
    if (o == Py_None) return otherwise;
    if (THPDtype_Check(o)) return reinterpret_cast<THPDtype*>(o)->scalar_type;
    const char* s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    require(s != nullptr);
    if (!std::strcmp(s, "bf16")) return at::ScalarType::BFloat16;
    if (!std::strcmp(s, "f16")) return at::ScalarType::Half;
    if (!std::strcmp(s, "f32")) return at::ScalarType::Float;
    throw Refused{};
}

// The launch, with other Python threads free to run.
template <typename F>
void run(F&& f) {
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = f();
    Py_END_ALLOW_THREADS
    require(status == TILES_OK);
}

PyObject* given(PyObject* o) {
    Py_INCREF(o);
    return o;
}

template <typename F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// x, weight, residual, eps, out, scales, h_out, stream, fp8 -> (y, scales, h)
PyObject* rmsnorm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        require(n == 9);
        const at::Tensor &x = tensor(args[0]), &weight = tensor(args[1]);
        const at::Tensor *residual = optional_tensor(args[2]), *out = optional_tensor(args[4]),
                         *scales = optional_tensor(args[5]), *h_out = optional_tensor(args[6]);
        const bool fp8 = args[8] == Py_True;
        const OnStream stream(args[7]);
        const Matrix mx(x);
        const at::ScalarType dtype = x.scalar_type(), out_dtype = fp8 ? kE4m3 : dtype;
        tiles_rmsnorm_desc d{};
        d.rows = mx.rows;
        d.cols = mx.cols;
        d.ldx = mx.ld;
        d.dtype = code_of(dtype);
        d.weight_dtype = code_of(weight.scalar_type());
        d.out_dtype = fp8 ? TILES_E4M3 : d.dtype;
        d.eps = number(args[3]);
        require(is_vector(weight, mx.cols, weight.scalar_type()));
        const int64_t nb = (mx.cols + 127) / 128;
        at::Tensor new_out, new_scales, new_h;
        if (out) {
            const Matrix m(*out);
            require(m.like(mx) && out->scalar_type() == out_dtype);
            d.ldy = m.ld;
        } else {
            // 8-bit rows: whole 16-byte pieces, as the products need.
            d.ldy = fp8 ? (mx.cols + 15) / 16 * 16 : mx.cols;
            new_out = empty_matrix(x, mx.rows, mx.cols, d.ldy, out_dtype);
            out = &new_out;
        }
        if (fp8) {
            if (scales) {
                require(scales->dim() == 2 && scales->size(0) == mx.rows && scales->size(1) == nb &&
                        scales->scalar_type() == at::ScalarType::Float);
            } else {
                new_scales = empty(x, {mx.rows, nb}, {1, mx.rows > 0 ? mx.rows : 1},
                                   at::ScalarType::Float);
                scales = &new_scales;
            }
            d.scale_row = scales->stride(0);
            d.scale_block = scales->stride(1);
            d.scales = static_cast<float*>(scales->data_ptr());
        }
        if (residual) {
            const Matrix m(*residual);
            require(m.like(mx) && residual->scalar_type() == dtype);
            d.residual = residual->data_ptr();
            d.ldr = m.ld;
            if (!h_out) {
                new_h = empty_matrix(x, mx.rows, mx.cols, mx.cols, dtype);
                h_out = &new_h;
            }
        }
        if (h_out) {
            const Matrix mh(*h_out);
            require(mh.like(mx) && h_out->scalar_type() == dtype);
            d.ldh = mh.ld;
            d.h = h_out->data_ptr();
        }
        d.x = x.data_ptr();
        d.weight = weight.data_ptr();
        d.y = out->data_ptr();
        run([&] { return calls.rmsnorm(&d, stream.at); });
        PyObject* h = new_h.defined() ? THPVariable_Wrap(std::move(new_h))
                                      : given(h_out ? args[6] : args[0]);
        PyObject* y = new_out.defined() ? THPVariable_Wrap(std::move(new_out)) : given(args[4]);
        PyObject* s = new_scales.defined() ? THPVariable_Wrap(std::move(new_scales)) : given(args[5]);
        PyObject* r = PyTuple_New(3);
        PyTuple_SET_ITEM(r, 0, y);
        PyTuple_SET_ITEM(r, 1, s);
        PyTuple_SET_ITEM(r, 2, h);
        return r;
    });
}

// dy, h, weight, eps, dh, dx_out, dweight_out, workspace, stream -> (dx, dweight)
PyObject* rmsnorm_grad(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        require(n == 9);
        const at::Tensor &dy = tensor(args[0]), &h = tensor(args[1]), &weight = tensor(args[2]);
        const at::Tensor *dh = optional_tensor(args[4]), *dx = optional_tensor(args[5]),
                         *dw = optional_tensor(args[6]);
        const OnStream stream(args[8]);
        const Matrix mh(h), mdy(dy);
        const at::ScalarType dtype = h.scalar_type();
        require(mdy.like(mh) && dy.scalar_type() == dtype &&
                is_vector(weight, mh.cols, weight.scalar_type()));
        tiles_rmsnorm_grad_desc d{};
        d.rows = mh.rows;
        d.cols = mh.cols;
        d.ldh = mh.ld;
        d.lddy = mdy.ld;
        d.dtype = code_of(dtype);
        d.weight_dtype = code_of(weight.scalar_type());
        d.eps = number(args[3]);
        if (dh) {
            const Matrix m(*dh);
            require(m.like(mh) && dh->scalar_type() == dtype);
            d.dh = dh->data_ptr();
            d.lddh = m.ld;
        }
        at::Tensor new_dx, new_dw;
        if (dx) {
            const Matrix m(*dx);
            require(m.like(mh) && dx->scalar_type() == dtype);
            d.lddx = m.ld;
        } else {
            d.lddx = mh.cols;
            new_dx = empty_matrix(h, mh.rows, mh.cols, mh.cols, dtype);
            dx = &new_dx;
        }
        if (dw) {
            require(is_vector(*dw, mh.cols, at::ScalarType::Float));
        } else {
            new_dw = empty(h, {mh.cols}, {1}, at::ScalarType::Float);
            dw = &new_dw;
        }
        d.dy = dy.data_ptr();
        d.h = h.data_ptr();
        d.weight = weight.data_ptr();
        d.dx = dx->data_ptr();
        d.dweight = static_cast<float*>(dw->data_ptr());
        const Workspace ws(args[7]);
        run([&] { return calls.rmsnorm_grad(&d, ws.at, ws.bytes, stream.at); });
        PyObject* r = PyTuple_New(2);
        PyTuple_SET_ITEM(r, 0, new_dx.defined() ? THPVariable_Wrap(std::move(new_dx)) : given(args[5]));
        PyTuple_SET_ITEM(r, 1, new_dw.defined() ? THPVariable_Wrap(std::move(new_dw)) : given(args[6]));
        return r;
    });
}

const int32_t* offsets_of(PyObject* o, int64_t groups) {
    const at::Tensor& t = tensor(o);
    require(groups >= 1 && is_vector(t, groups + 1, at::ScalarType::Int));
    return static_cast<const int32_t*>(t.data_ptr());
}

// The output of a product: given, or new.
const at::Tensor* product_out(const at::Tensor* out, at::Tensor* made, const at::Tensor& like,
                              tiles_product_desc* d, PyObject* dtype, at::ScalarType otherwise) {
    if (out) {
        const Matrix m(*out);
        require(m.rows == d->m && m.cols == d->n);
        d->ldc = m.ld;
    } else {
        d->ldc = d->n;
        const at::ScalarType t = out_type(dtype, otherwise);
        code_of(t);
        *made = empty_matrix(like, d->m, d->n, d->n, t);
        out = made;
    }
    d->out_dtype = code_of(out->scalar_type());
    d->c = out->data_ptr();
    return out;
}

// a, a_scales, b, b_scales, offsets or None, out, out_dtype, workspace, stream -> out
PyObject* product_fp8(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        require(n == 9);
        const at::Tensor &a = tensor(args[0]), &as = tensor(args[1]), &b = tensor(args[2]),
                         &bs = tensor(args[3]);
        const bool grouped = args[4] != Py_None;
        const OnStream stream(args[8]);
        const Matrix ma(a);
        const Weight mb(b, grouped);
        tiles_product_desc d{};
        d.m = ma.rows;
        d.n = mb.rows;
        d.k = ma.cols;
        d.groups = mb.groups;
        if (grouped) d.offsets = offsets_of(args[4], mb.groups);
        const int64_t kb = (d.k + 127) / 128, nb = (d.n + 127) / 128;
        const int g = grouped ? 1 : 0;
        require(mb.cols == d.k && a.scalar_type() == kE4m3 && b.scalar_type() == kE4m3 &&
                as.dim() == 2 && as.size(0) == d.m && as.size(1) == kb && bs.dim() == 2 + g &&
                bs.size(g) == nb && bs.size(g + 1) == kb && (!grouped || bs.size(0) == mb.groups) &&
                as.scalar_type() == at::ScalarType::Float && bs.scalar_type() == at::ScalarType::Float);
        at::Tensor made;
        product_out(optional_tensor(args[5]), &made, a, &d, args[6], at::ScalarType::BFloat16);
        d.a = a.data_ptr();
        d.b = b.data_ptr();
        d.a_scales = static_cast<const float*>(as.data_ptr());
        d.b_scales = static_cast<const float*>(bs.data_ptr());
        d.lda = ma.ld;
        d.ldb = mb.ld;
        d.stride_b = mb.stride;
        d.a_scale_row = as.stride(0);
        d.a_scale_block = as.stride(1);
        d.b_scale_row = bs.stride(g);
        d.b_scale_block = bs.stride(g + 1);
        d.b_scale_group = grouped ? bs.stride(0) : 0;
        d.in_dtype = TILES_E4M3;
        d.b_layout = TILES_B_NK;
        const Workspace ws(args[7]);
        run([&] { return (grouped ? calls.grouped_gemm : calls.gemm_fp8)(&d, ws.at, ws.bytes, stream.at); });
        return made.defined() ? THPVariable_Wrap(std::move(made)) : given(args[5]);
    });
}

// a, b, offsets, trans_b, out, out_dtype, workspace, stream -> out
PyObject* grouped_gemm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        require(n == 8 && PyBool_Check(args[3]));
        const at::Tensor &a = tensor(args[0]), &b = tensor(args[1]);
        const bool trans = args[3] == Py_True;
        const OnStream stream(args[7]);
        const Matrix ma(a);
        const Weight mb(b, true);
        const at::ScalarType dtype = a.scalar_type();
        tiles_product_desc d{};
        d.m = ma.rows;
        d.n = trans ? mb.rows : mb.cols;
        d.k = ma.cols;
        d.groups = mb.groups;
        d.offsets = offsets_of(args[2], mb.groups);
        d.in_dtype = code_of(dtype);
        require((trans ? mb.cols : mb.rows) == d.k && b.scalar_type() == dtype);
        at::Tensor made;
        product_out(optional_tensor(args[4]), &made, a, &d, args[5], dtype);
        d.a = a.data_ptr();
        d.b = b.data_ptr();
        d.lda = ma.ld;
        d.ldb = mb.ld;
        d.stride_b = mb.stride;
        d.b_layout = trans ? TILES_B_NK : TILES_B_KN;
        const Workspace ws(args[6]);
        run([&] { return calls.grouped_gemm(&d, ws.at, ws.bytes, stream.at); });
        return made.defined() ? THPVariable_Wrap(std::move(made)) : given(args[4]);
    });
}

// a, dc, offsets, out, out_dtype, workspace, stream -> out
PyObject* grouped_wgrad(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        require(n == 7);
        const at::Tensor &a = tensor(args[0]), &dc = tensor(args[1]), &off = tensor(args[2]);
        const at::Tensor* out = optional_tensor(args[3]);
        const OnStream stream(args[6]);
        const Matrix ma(a), mc(dc);
        const at::ScalarType dtype = a.scalar_type();
        require(mc.rows == ma.rows && dc.scalar_type() == dtype && off.dim() == 1);
        tiles_wgrad_desc d{};
        d.m = ma.rows;
        d.k = ma.cols;
        d.n = mc.cols;
        d.groups = off.size(0) - 1;
        d.offsets = offsets_of(args[2], d.groups);
        d.in_dtype = code_of(dtype);
        at::Tensor made;
        if (out) {
            const Weight m(*out, true);
            require(m.groups == d.groups && m.rows == d.k && m.cols == d.n);
            d.lddw = m.ld;
            d.stride_dw = m.stride;
        } else {
            const at::ScalarType t = out_type(args[4], dtype);
            code_of(t);
            d.lddw = d.n;
            d.stride_dw = d.k * d.n;
            made = empty(a, {d.groups, d.k, d.n}, {d.stride_dw, d.n, 1}, t);
            out = &made;
        }
        d.out_dtype = code_of(out->scalar_type());
        d.a = a.data_ptr();
        d.dc = dc.data_ptr();
        d.dw = out->data_ptr();
        d.lda = ma.ld;
        d.lddc = mc.ld;
        const Workspace ws(args[5]);
        run([&] { return calls.grouped_wgrad(&d, ws.at, ws.bytes, stream.at); });
        return made.defined() ? THPVariable_Wrap(std::move(made)) : given(args[3]);
    });
}

// A call's workspace: the caller's, or memory of the call's own from the current
// stream's pool (call under OnStream), which goes back there when the call is
// made: whatever takes it next on the stream runs after the call's kernels.
struct Scratch {
    static constexpr size_t kHeader = 256;
    Workspace given;
    at::Tensor own;

    Scratch(PyObject* o, size_t bytes, const at::Tensor& like) : given(o) {
        require(bytes > 0);
        if (given.at || bytes <= kHeader) return;  // no more than the header: nothing is used
        own = empty(like, {static_cast<int64_t>(bytes)}, {1}, at::ScalarType::Byte);
        given.at = own.data_ptr();
        given.bytes = bytes;
    }
};

// Autograd learns what a call has written into the caller's tensor, as of any
// operation in place.  (It never throws: the call has been made.)
void wrote(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject* written(PyObject* arg) {
    if (arg != Py_None) wrote(THPVariable_Unpack(arg));
    return given(arg);
}

// A new output, or the caller's argument.
PyObject* made_or(at::Tensor& made, PyObject* arg) {
    return made.defined() ? THPVariable_Wrap(std::move(made)) : written(arg);
}

// x, weight, bias, residual, eps, out, scales, h_out, stream, fp8 -> (y, scales, h)
PyObject* layernorm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        require(n == 10);
        const at::Tensor &x = tensor(args[0]), &weight = tensor(args[1]);
        const at::Tensor *bias = optional_tensor(args[2]), *residual = optional_tensor(args[3]),
                         *out = optional_tensor(args[5]), *scales = optional_tensor(args[6]),
                         *h_out = optional_tensor(args[7]);
        const bool fp8 = args[9] == Py_True;
        const OnStream stream(args[8]);
        const Matrix mx(x);
        const at::ScalarType dtype = x.scalar_type(), out_dtype = fp8 ? kE4m3 : dtype;
        tiles_layernorm_desc d{};
        d.rows = mx.rows;
        d.cols = mx.cols;
        d.ldx = mx.ld;
        d.dtype = code_of(dtype);
        d.weight_dtype = code_of(weight.scalar_type());
        d.out_dtype = fp8 ? TILES_E4M3 : d.dtype;
        d.eps = number(args[4]);
        require(is_vector(weight, mx.cols, weight.scalar_type()) &&
                (!bias || is_vector(*bias, mx.cols, weight.scalar_type())));
        at::Tensor new_out, new_scales, new_h;
        if (out) {
            const Matrix m(*out);
            require(m.like(mx) && out->scalar_type() == out_dtype);
            d.ldy = m.ld;
        } else {
            d.ldy = fp8 ? (mx.cols + 15) / 16 * 16 : mx.cols;
            new_out = empty_matrix(x, mx.rows, mx.cols, d.ldy, out_dtype);
            out = &new_out;
        }
        if (fp8) {
            const int64_t nb = (mx.cols + 127) / 128;
            if (scales) {
                require(scales->dim() == 2 && scales->size(0) == mx.rows && scales->size(1) == nb &&
                        scales->scalar_type() == at::ScalarType::Float);
            } else {
                new_scales = empty(x, {mx.rows, nb}, {1, mx.rows > 0 ? mx.rows : 1},
                                   at::ScalarType::Float);
                scales = &new_scales;
            }
            d.scale_row = scales->stride(0);
            d.scale_block = scales->stride(1);
            d.scales = static_cast<float*>(scales->data_ptr());
        }
        if (residual) {
            const Matrix m(*residual);
            require(m.like(mx) && residual->scalar_type() == dtype);
            d.residual = residual->data_ptr();
            d.ldr = m.ld;
            if (!h_out) {
                new_h = empty_matrix(x, mx.rows, mx.cols, mx.cols, dtype);
                h_out = &new_h;
            }
        }
        if (h_out) {
            const Matrix mh(*h_out);
            require(mh.like(mx) && h_out->scalar_type() == dtype);
            d.ldh = mh.ld;
            d.h = h_out->data_ptr();
        }
        d.x = x.data_ptr();
        d.weight = weight.data_ptr();
        d.bias = bias ? bias->data_ptr() : nullptr;
        d.y = out->data_ptr();
        run([&] { return calls.layernorm(&d, stream.at); });
        PyObject* h = new_h.defined() ? THPVariable_Wrap(std::move(new_h))
                                      : h_out ? written(args[7]) : given(args[0]);
        PyObject* r = PyTuple_New(3);
        PyTuple_SET_ITEM(r, 0, made_or(new_out, args[5]));
        PyTuple_SET_ITEM(r, 1, made_or(new_scales, args[6]));
        PyTuple_SET_ITEM(r, 2, h);
        return r;
    });
}

// dy, h, weight, eps, dh, dx_out, dweight_out, dbias_out, workspace, stream
// -> (dx, dweight, dbias)
PyObject* layernorm_grad(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        require(n == 10);
        const at::Tensor &dy = tensor(args[0]), &h = tensor(args[1]), &weight = tensor(args[2]);
        const at::Tensor *dh = optional_tensor(args[4]), *dx = optional_tensor(args[5]);
        const OnStream stream(args[9]);
        const Matrix mh(h), mdy(dy);
        const at::ScalarType dtype = h.scalar_type();
        require(mdy.like(mh) && dy.scalar_type() == dtype &&
                is_vector(weight, mh.cols, weight.scalar_type()));
        tiles_layernorm_grad_desc d{};
        d.rows = mh.rows;
        d.cols = mh.cols;
        d.ldh = mh.ld;
        d.lddy = mdy.ld;
        d.dtype = code_of(dtype);
        d.weight_dtype = code_of(weight.scalar_type());
        d.eps = number(args[3]);
        if (dh) {
            const Matrix m(*dh);
            require(m.like(mh) && dh->scalar_type() == dtype);
            d.dh = dh->data_ptr();
            d.lddh = m.ld;
        }
        at::Tensor new_dx, new_sum[2];
        if (dx) {
            const Matrix m(*dx);
            require(m.like(mh) && dx->scalar_type() == dtype);
            d.lddx = m.ld;
        } else {
            d.lddx = mh.cols;
            new_dx = empty_matrix(h, mh.rows, mh.cols, mh.cols, dtype);
            dx = &new_dx;
        }
        float* sums[2];
        for (int i = 0; i < 2; ++i) {
            const at::Tensor* t = optional_tensor(args[6 + i]);
            if (t) {
                require(is_vector(*t, mh.cols, at::ScalarType::Float));
            } else {
                new_sum[i] = empty(h, {mh.cols}, {1}, at::ScalarType::Float);
                t = &new_sum[i];
            }
            sums[i] = static_cast<float*>(t->data_ptr());
        }
        d.dy = dy.data_ptr();
        d.h = h.data_ptr();
        d.weight = weight.data_ptr();
        d.dx = dx->data_ptr();
        d.dweight = sums[0];
        d.dbias = sums[1];
        const Scratch ws(args[8], calls.layernorm_grad_workspace_bytes(d.rows, d.cols), h);
        run([&] { return calls.layernorm_grad(&d, ws.given.at, ws.given.bytes, stream.at); });
        PyObject* r = PyTuple_New(3);
        PyTuple_SET_ITEM(r, 0, made_or(new_dx, args[5]));
        PyTuple_SET_ITEM(r, 1, made_or(new_sum[0], args[6]));
        PyTuple_SET_ITEM(r, 2, made_or(new_sum[1], args[7]));
        return r;
    });
}

// experts, groups, workspace, stream -> (slots, offsets, order)
PyObject* expert_sort(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        require(n == 4);
        const at::Tensor& experts = tensor(args[0]);
        const OnStream stream(args[3]);
        const Matrix m(experts);
        const at::ScalarType dtype = experts.scalar_type();
        require(dtype == at::ScalarType::Int || dtype == at::ScalarType::Long);
        tiles_expert_sort_desc d{};
        d.tokens = m.rows;
        d.k = m.cols;
        d.groups = PyLong_AsLongLong(args[1]);
        require(!PyErr_Occurred());
        d.experts = experts.data_ptr();
        d.ld = m.ld;
        d.index_bytes = dtype == at::ScalarType::Long ? 8 : 4;
        const Scratch ws(args[2], calls.expert_sort_workspace_bytes(d.tokens, d.k, d.groups), experts);
        const auto type = at::ScalarType::Int;
        at::Tensor slots = empty_matrix(experts, m.rows, m.cols, m.cols, type);
        at::Tensor offsets = empty(experts, {d.groups + 1}, {1}, type);
        at::Tensor order = empty(experts, {m.rows * m.cols}, {1}, type);
        d.slots = static_cast<int32_t*>(slots.data_ptr());
        d.offsets = static_cast<int32_t*>(offsets.data_ptr());
        d.order = static_cast<int32_t*>(order.data_ptr());
        run([&] { return calls.expert_sort(&d, ws.given.at, ws.given.bytes, stream.at); });
        PyObject* r = PyTuple_New(3);
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(slots)));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(offsets)));
        PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(order)));
        return r;
    });
}

// The slots of `tokens` tokens (any number where tokens < 0).
Matrix slots_of(const at::Tensor& t, int64_t tokens) {
    const Matrix m(t);
    require(t.scalar_type() == at::ScalarType::Int && (tokens < 0 || m.rows == tokens));
    return m;
}

// x, slots, scales, out, scales_out, stream -> out, or (out, scales)
PyObject* expert_dispatch(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        require(n == 6);
        const at::Tensor &x = tensor(args[0]), &slots = tensor(args[1]);
        const at::Tensor *scales = optional_tensor(args[2]), *out = optional_tensor(args[3]),
                         *scales_out = optional_tensor(args[4]);
        const OnStream stream(args[5]);
        const Matrix mx(x), ms = slots_of(slots, mx.rows);
        const at::ScalarType dtype = x.scalar_type();
        const bool fp8 = dtype == kE4m3;
        tiles_dispatch_desc d{};
        d.tokens = mx.rows;
        d.cols = mx.cols;
        d.k = ms.cols;
        d.ldx = mx.ld;
        d.ld_slots = ms.ld;
        d.dtype = fp8 ? TILES_E4M3 : code_of(dtype);
        at::Tensor new_out, new_scales;
        if (out) {
            const Matrix m(*out);
            require(m.cols == mx.cols && out->scalar_type() == dtype);
            d.rows = m.rows;
            d.ld_out = m.ld;
        } else {
            d.rows = d.tokens * d.k;
            d.ld_out = fp8 ? (mx.cols + 15) / 16 * 16 : mx.cols;
            new_out = empty_matrix(x, d.rows, mx.cols, d.ld_out, dtype);
            out = &new_out;
        }
        require(scales || !scales_out);
        if (scales) {
            const int64_t nb = (mx.cols + 127) / 128;
            if (!scales_out) {
                new_scales = empty(x, {d.rows, nb}, {1, d.rows > 0 ? d.rows : 1}, at::ScalarType::Float);
                scales_out = &new_scales;
            }
            require(scales->dim() == 2 && scales->size(0) == d.tokens && scales->size(1) == nb &&
                    scales->scalar_type() == at::ScalarType::Float && scales_out->dim() == 2 &&
                    scales_out->size(0) == d.rows && scales_out->size(1) == nb &&
                    scales_out->scalar_type() == at::ScalarType::Float);
            d.scales = static_cast<const float*>(scales->data_ptr());
            d.out_scales = static_cast<float*>(scales_out->data_ptr());
            d.scale_row = scales->stride(0);
            d.scale_block = scales->stride(1);
            d.out_scale_row = scales_out->stride(0);
            d.out_scale_block = scales_out->stride(1);
        }
        d.x = x.data_ptr();
        d.slots = static_cast<const int32_t*>(slots.data_ptr());
        d.out = out->data_ptr();
        run([&] { return calls.expert_dispatch(&d, stream.at); });
        if (!scales) return made_or(new_out, args[3]);
        PyObject* r = PyTuple_New(2);
        PyTuple_SET_ITEM(r, 0, made_or(new_out, args[3]));
        PyTuple_SET_ITEM(r, 1, made_or(new_scales, args[4]));
        return r;
    });
}

// What the sum and its gradients have in common.
tiles_combine_desc combine_of(const at::Tensor& rows, const at::Tensor& slots,
                              const at::Tensor* weights) {
    const Matrix mr(rows), ms = slots_of(slots, -1);
    tiles_combine_desc d{};
    d.tokens = ms.rows;
    d.k = ms.cols;
    d.rows = mr.rows;
    d.cols = mr.cols;
    d.ld_slots = ms.ld;
    d.ld_in = mr.ld;
    d.dtype = code_of(rows.scalar_type());
    d.slots = static_cast<const int32_t*>(slots.data_ptr());
    d.in = rows.data_ptr();
    if (weights) {
        const Matrix m(*weights);
        require(m.like(ms));
        d.weights = weights->data_ptr();
        d.ld_weights = m.ld;
        d.weight_dtype = code_of(weights->scalar_type());
    }
    return d;
}

// rows, slots, weights, out, stream -> out
PyObject* expert_combine(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        require(n == 5);
        const at::Tensor& rows = tensor(args[0]);
        const at::Tensor* out = optional_tensor(args[3]);
        const OnStream stream(args[4]);
        tiles_combine_desc d = combine_of(rows, tensor(args[1]), optional_tensor(args[2]));
        at::Tensor made;
        if (out) {
            const Matrix m(*out);
            require(m.rows == d.tokens && m.cols == d.cols && out->scalar_type() == rows.scalar_type());
            d.ld_out = m.ld;
        } else {
            d.ld_out = d.cols;
            made = empty_matrix(rows, d.tokens, d.cols, d.cols, rows.scalar_type());
            out = &made;
        }
        d.out = out->data_ptr();
        run([&] { return calls.expert_combine(&d, stream.at); });
        return made_or(made, args[3]);
    });
}

// dy, rows, slots, weights, drows_out, dweights_out, stream -> (drows, dweights)
PyObject* expert_combine_grad(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        require(n == 7);
        const at::Tensor &dy = tensor(args[0]), &rows = tensor(args[1]), &weights = tensor(args[3]);
        const at::Tensor *drows = optional_tensor(args[4]), *dweights = optional_tensor(args[5]);
        const OnStream stream(args[6]);
        tiles_combine_desc d = combine_of(rows, tensor(args[2]), &weights);
        const Matrix mdy(dy);
        const at::ScalarType dtype = rows.scalar_type();
        require(mdy.rows == d.tokens && mdy.cols == d.cols && dy.scalar_type() == dtype);
        d.dy = dy.data_ptr();
        d.ld_dy = mdy.ld;
        at::Tensor new_rows, new_weights;
        if (drows) {
            const Matrix m(*drows);
            require(m.rows == d.rows && m.cols == d.cols && drows->scalar_type() == dtype);
            d.ld_out = m.ld;
        } else {
            d.ld_out = d.cols;
            new_rows = empty_matrix(rows, d.rows, d.cols, d.cols, dtype);
            drows = &new_rows;
        }
        if (dweights) {
            const Matrix m(*dweights);
            require(m.rows == d.tokens && m.cols == d.k && dweights->scalar_type() == at::ScalarType::Float);
            d.ld_dweights = m.ld;
        } else {
            d.ld_dweights = d.k;
            new_weights = empty_matrix(rows, d.tokens, d.k, d.k, at::ScalarType::Float);
            dweights = &new_weights;
        }
        d.out = drows->data_ptr();
        d.dweights = static_cast<float*>(dweights->data_ptr());
        run([&] { return calls.expert_combine_grad(&d, stream.at); });
        PyObject* r = PyTuple_New(2);
        PyTuple_SET_ITEM(r, 0, made_or(new_rows, args[4]));
        PyTuple_SET_ITEM(r, 1, made_or(new_weights, args[5]));
        return r;
    });
}

// grads (a list), max_norm (None: the norm alone), eps, out (a list or None),
// workspace, stream -> norm
PyObject* clip_grads(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        require(n == 6 && PyList_Check(args[0]) && (args[3] == Py_None || PyList_Check(args[3])));
        const Py_ssize_t count = PyList_GET_SIZE(args[0]);
        const bool apart = args[3] != Py_None;
        require(count > 0 && (!apart || PyList_GET_SIZE(args[3]) == count));
        const OnStream stream(args[5]);
        std::vector<tiles_grad_tensor> tensors(static_cast<size_t>(count));
        for (Py_ssize_t i = 0; i < count; ++i) {
            const at::Tensor& g = tensor(PyList_GET_ITEM(args[0], i));
            require(g.is_non_overlapping_and_dense());
            tiles_grad_tensor& t = tensors[static_cast<size_t>(i)];
            t = {g.data_ptr(), nullptr, g.numel(), code_of(g.scalar_type()), 0};
            if (apart) {
                const at::Tensor& o = tensor(PyList_GET_ITEM(args[3], i));
                require(o.scalar_type() == g.scalar_type() && o.sizes() == g.sizes() &&
                        o.strides() == g.strides());
                t.out = o.data_ptr();
            }
        }
        const at::Tensor& like = tensor(PyList_GET_ITEM(args[0], 0));
        const Scratch ws(args[4], calls.grad_norm_workspace_bytes(count), like);
        at::Tensor norm = empty(like, {}, {}, at::ScalarType::Float);
        float* at = static_cast<float*>(norm.data_ptr());
        if (args[1] == Py_None) {
            run([&] { return calls.grad_norm(tensors.data(), count, at, ws.given.at, ws.given.bytes, stream.at); });
        } else {
            const float max_norm = number(args[1]), eps = number(args[2]);
            run([&] {
                return calls.clip_grads(tensors.data(), count, max_norm, eps, at, ws.given.at,
                                        ws.given.bytes, stream.at);
            });
            PyObject* const to = apart ? args[3] : args[0];
            for (Py_ssize_t i = 0; i < count; ++i) wrote(THPVariable_Unpack(PyList_GET_ITEM(to, i)));
        }
        return THPVariable_Wrap(std::move(norm));
    });
}

// The addresses, in the order of Calls.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    constexpr int kCalls = sizeof(calls) / sizeof(void*);
    if (n != kCalls) {
        PyErr_Format(PyExc_TypeError, "bind takes %d addresses", kCalls);
        return nullptr;
    }
    void* at[kCalls];
    for (int i = 0; i < kCalls; ++i) {
        at[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    std::memcpy(&calls, at, sizeof(at));
    Py_RETURN_NONE;
}

#define TILES_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TILES_METHOD(bind), TILES_METHOD(rmsnorm), TILES_METHOD(rmsnorm_grad),
                         TILES_METHOD(product_fp8), TILES_METHOD(grouped_gemm),
                         TILES_METHOD(grouped_wgrad), TILES_METHOD(layernorm),
                         TILES_METHOD(layernorm_grad), TILES_METHOD(expert_sort),
                         TILES_METHOD(expert_dispatch), TILES_METHOD(expert_combine),
                         TILES_METHOD(expert_combine_grad), TILES_METHOD(clip_grads), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__calls() { return PyModule_Create(&module); }
