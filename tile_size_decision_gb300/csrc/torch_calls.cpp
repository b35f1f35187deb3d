// The short calls on PyTorch tensors (norms, 8-bit and grouped products), as a
// Python module.  A decoding step's norm or product takes a few microseconds
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

// The five addresses, in the order of Calls.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
        return nullptr;
    }
    void* at[5];
    for (int i = 0; i < 5; ++i) {
        at[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    static_assert(sizeof(calls) == sizeof(at), "one address a call");
    std::memcpy(&calls, at, sizeof(at));
    Py_RETURN_NONE;
}

#define TILES_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TILES_METHOD(bind), TILES_METHOD(rmsnorm), TILES_METHOD(rmsnorm_grad),
                         TILES_METHOD(product_fp8), TILES_METHOD(grouped_gemm),
                         TILES_METHOD(grouped_wgrad), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__calls() { return PyModule_Create(&module); }
