// python_ops.cpp -- the compiled half of the Python binding of the operators around the routed layer
// (operators.py has the public functions): checks of the tensors, allocation of the outputs, one call of the C ABI.
//
// A small call is over on the GPU in two or three microseconds.  Through ctypes and Python's tensor methods the
// way there cost 8 to 11 us of host time a call; here it is the launch and little else.
//
// Every function takes its arguments by position, None for an absent tensor, enqueues on the current stream of
// the tensors' device and returns the outputs.  What the C ABI refuses raises the exception class that operators.py
// hands over (raise_as).
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>

#include "moe.h"

namespace {

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kI8 = at::kChar, kI32 = at::kInt;

// A tensor argument that did not fit; becomes a ValueError (TypeError if it is no tensor).
struct Refusal {
    PyObject *type;
    std::string text;
};

std::string describe(const at::Tensor &t)
{
    std::ostringstream s;
    s << toString(t.scalar_type()) << " [";
    for (int64_t i = 0; i < t.dim(); ++i) s << (i ? ", " : "") << t.size(i);
    s << "] on " << t.device() << (t.is_contiguous() ? "" : " (strided)");
    return s.str();
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) throw Refusal{PyExc_TypeError, std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}

[[noreturn]] void refuse(const at::Tensor &t, const char *name, at::ScalarType type, const std::string &shape)
{
    throw Refusal{PyExc_ValueError, std::string(name) + " must be a contiguous CUDA tensor of " + toString(type) + " " +
                                        shape + " on the call's device, got " + describe(t)};
}

// The tensor whose device the call runs on.
const at::Tensor &lead(PyObject *o, const char *name, at::ScalarType type)
{
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || !t.is_cuda() || t.dim() != 2 || !t.is_contiguous()) refuse(t, name, type, "[rows, columns]");
    return t;
}

// Address of a tensor that has to have this type and shape; nullptr for None if `optional`.
void *address(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, const at::Device &dev,
              bool optional = false)
{
    if (optional && o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || t.device() != dev || t.sizes() != shape || !t.is_contiguous()) {
        std::ostringstream s;
        s << shape;
        refuse(t, name, type, s.str());
    }
    return t.data_ptr();
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Device &dev)
{
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

// Two new outputs.  Small ones share an allocation, the second 512 bytes or a multiple of that into it: an allocation
// costs 0.8 us of host time, a fifth of a small call.  Larger ones have their own, so that neither keeps the other's
// memory.
constexpr size_t kSharedBytes = 1 << 20;   // what the allocator hands out as small blocks
void make_two(at::Tensor &a, at::IntArrayRef a_shape, at::ScalarType a_type, at::Tensor &b, at::IntArrayRef b_shape,
              at::ScalarType b_type, const at::Device &dev)
{
    auto bytes = [](at::IntArrayRef shape, at::ScalarType type) {
        return static_cast<size_t>(c10::multiply_integers(shape)) * c10::elementSize(type);
    };
    const size_t a_bytes = (bytes(a_shape, a_type) + 511) / 512 * 512, total = a_bytes + bytes(b_shape, b_type);
    if (total == 0 || total > kSharedBytes) {
        a = make(a_shape, a_type, dev);
        b = make(b_shape, b_type, dev);
        return;
    }
    c10::Allocator *from = c10::cuda::CUDACachingAllocator::get();
    const c10::Storage both(c10::Storage::use_byte_size_t(), total, from->allocate(total), from, /*resizable=*/false);
    auto part = [&](at::IntArrayRef shape, at::ScalarType type, size_t offset) {
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(both), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                                c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
        t.unsafeGetTensorImpl()->set_storage_offset(static_cast<int64_t>(offset / c10::elementSize(type)));
        return t;
    };
    a = part(a_shape, a_type, 0);
    b = part(b_shape, b_type, a_bytes);
}

// The caller's output tensor, or a new one.
at::Tensor output(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, const at::Device &dev)
{
    if (o == Py_None) return make(shape, type, dev);
    address(o, name, type, shape, dev);
    return THPVariable_Unpack(o);
}

// For the C ABI, which takes int sizes: larger ones are refused there as unsupported, not cut off here.
int size(int64_t v) { return v > 0x7fffffff ? 0x7fffffff : static_cast<int>(v); }

// The call's device and its current stream.
struct Place {
    c10::cuda::CUDAGuard guard;
    cudaStream_t stream;
    explicit Place(const at::Device &dev) : guard(dev), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream()) {}
};

PyObject *wrap_all(std::initializer_list<const at::Tensor *> all)
{
    PyObject *tuple = PyTuple_New(static_cast<Py_ssize_t>(all.size()));
    if (!tuple) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor *t : all) {
        PyObject *o = nullptr;
        if (t->defined()) {
            o = THPVariable_Wrap(*t);
        } else {
            o = Py_None;
            Py_INCREF(o);
        }
        if (!o) {
            Py_DECREF(tuple);
            return nullptr;
        }
        PyTuple_SET_ITEM(tuple, i++, o);
    }
    return tuple;
}

float real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return static_cast<float>(v);
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

long long whole(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

PyObject *error_class = nullptr;   // called as error_class(status, function)

PyObject *failed(int status, const char *function)
{
    PyObject *e = error_class ? PyObject_CallFunction(error_class, "is", status, function) : nullptr;
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
        PyErr_Format(PyExc_RuntimeError, "%s returned %d", function, status);
    }
    return nullptr;
}

PyObject *raise_as(PyObject *, PyObject *cls)
{
    Py_INCREF(cls);
    Py_XSETREF(error_class, cls);
    Py_RETURN_NONE;
}

PyObject *count_error(const char *name, Py_ssize_t want, Py_ssize_t got)
{
    return PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
}

#define MOE_BEGIN(name, want)                                  \
    HANDLE_TH_ERRORS                                           \
    if (n != (want)) return count_error(name, (want), n);      \
    try {
#define MOE_END                                                \
    }                                                          \
    catch (const Refusal &r)                                   \
    {                                                          \
        PyErr_SetString(r.type, r.text.c_str());               \
        return nullptr;                                        \
    }                                                          \
    END_HANDLE_TH_ERRORS

// (x, residual, w_post, gate, w_pre, eps, residual_scale, block_scale, w_offset, quantize, res_out, h_out)
PyObject *block_norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    MOE_BEGIN("block_norm", 12)
    const at::Tensor &x = lead(a[0], "x", kBf16);
    const at::Device dev = x.device();
    const Place place(dev);
    const int64_t M = x.size(0), H = x.size(1);
    const void *residual = address(a[1], "residual", kBf16, {M, H}, dev, true);
    const void *w_post = address(a[2], "w_post", kBf16, {H}, dev, true);
    const void *w_pre = address(a[4], "w_pre", kBf16, {H}, dev, true);
    const void *gate = nullptr;
    int kind = MOE_GATE_NONE;
    if (a[3] != Py_None) {
        const at::Tensor &g = tensor(a[3], "gate");
        if (g.scalar_type() == kF32) {
            kind = MOE_GATE_TOKEN;
            gate = g.dim() == 2 ? address(a[3], "gate", kF32, {M, 1}, dev) : address(a[3], "gate", kF32, {M}, dev);
        } else if (g.dim() == 1) {
            kind = MOE_GATE_CHANNEL;
            gate = address(a[3], "gate", kBf16, {H}, dev);
        } else {
            kind = MOE_GATE_FULL;
            gate = address(a[3], "gate", kBf16, {M, H}, dev);
        }
    }
    const float eps = real(a[5]), residual_scale = real(a[6]), block_scale = real(a[7]), w_offset = real(a[8]);
    const bool quantize = truth(a[9]), has_pre = a[4] != Py_None;
    if (!has_pre && (quantize || a[11] != Py_None)) throw Refusal{PyExc_ValueError, "h and its codes need w_pre"};
    at::Tensor r, h, q, q_s;
    const bool changes = a[1] != Py_None || a[2] != Py_None || a[3] != Py_None || !has_pre || block_scale != 1.0f;
    if (changes && has_pre && a[10] == Py_None && a[11] == Py_None) {
        make_two(r, {M, H}, kBf16, h, {M, H}, kBf16, dev);
    } else {
        if (changes || a[10] != Py_None) r = output(a[10], "res_out", kBf16, {M, H}, dev);
        if (has_pre) h = output(a[11], "h_out", kBf16, {M, H}, dev);
    }
    if (quantize) make_two(q, {M, H}, kI8, q_s, {M}, kF32, dev);
    auto at_of = [](const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
    const int rc = moe_block_norm(x.data_ptr(), residual, w_post, gate, kind, w_pre, block_scale, residual_scale, eps,
                                  w_offset, at_of(r), at_of(h), static_cast<int8_t *>(at_of(q)),
                                  static_cast<float *>(at_of(q_s)), size(M), size(H), place.stream);
    if (rc != MOE_OK) return failed(rc, "moe_block_norm");
    return quantize ? wrap_all({&r, &h, &q, &q_s}) : wrap_all({&r, &h});
    MOE_END
}

// (x, swiglu)
PyObject *int8_quantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    MOE_BEGIN("int8_quantize", 2)
    const at::Tensor &x = lead(a[0], "x", kBf16);
    const at::Device dev = x.device();
    const Place place(dev);
    const bool swiglu = truth(a[1]);
    const int64_t M = x.size(0), K = swiglu ? x.size(1) / 2 : x.size(1);
    if (swiglu && x.size(1) % 2) throw Refusal{PyExc_ValueError, "x must hold as many gate as up columns"};
    at::Tensor q, s;
    make_two(q, {M, K}, kI8, s, {M}, kF32, dev);
    const int rc = moe_int8_quantize(x.data_ptr(), swiglu, static_cast<int8_t *>(q.data_ptr()),
                                     static_cast<float *>(s.data_ptr()), size(M), size(K), place.stream);
    if (rc != MOE_OK) return failed(rc, "moe_int8_quantize");
    return wrap_all({&q, &s});
    MOE_END
}

// (q, q_s, w_q, w_s, add, out, out_f32, status_out)
PyObject *int8_gemm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    MOE_BEGIN("int8_gemm", 8)
    const at::Tensor &q = lead(a[0], "q", kI8);
    const at::Device dev = q.device();
    const Place place(dev);
    const at::Tensor &w = tensor(a[2], "w_q");
    const int64_t M = q.size(0), K = q.size(1), N = w.dim() == 2 ? w.size(0) : -1;
    const void *w_q = address(a[2], "w_q", kI8, {N, K}, dev);
    const void *q_s = address(a[1], "q_s", kF32, {M}, dev), *w_s = address(a[3], "w_s", kF32, {N}, dev);
    const void *add = address(a[4], "add", kBf16, {M, N}, dev, true);
    void *status = address(a[7], "status_out", kI32, {1}, dev, true);
    const bool f32 = truth(a[6]);
    const at::Tensor out = output(a[5], "out", f32 ? kF32 : kBf16, {M, N}, dev);
    const int rc = moe_int8_gemm(static_cast<const int8_t *>(q.data_ptr()), static_cast<const float *>(q_s),
                                 static_cast<const int8_t *>(w_q), static_cast<const float *>(w_s), add, out.data_ptr(),
                                 f32, size(M), size(N), size(K), static_cast<int32_t *>(status), place.stream);
    if (rc != MOE_OK) return failed(rc, "moe_int8_gemm");
    return THPVariable_Wrap(out);
    MOE_END
}

// (x, w, expert_offsets, sorted_ids, k, swiglu, out, out_f32, status_out)
PyObject *grouped_gemm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    MOE_BEGIN("grouped_gemm", 9)
    const at::Tensor &x = lead(a[0], "x", kBf16);
    const at::Device dev = x.device();
    const Place place(dev);
    const at::Tensor &w = tensor(a[1], "w");
    const bool swiglu = truth(a[5]), f32 = truth(a[7]);
    const int64_t M = x.size(0), K = x.size(1), E = w.dim() == 3 ? w.size(0) : -1, rows = w.dim() == 3 ? w.size(1) : -1;
    const void *wp = address(a[1], "w", kBf16, {E, rows, K}, dev);
    if (swiglu && rows % 2) throw Refusal{PyExc_ValueError, "w must hold as many gate as up rows"};
    const int64_t N = swiglu ? rows / 2 : rows;
    const void *offsets = address(a[2], "expert_offsets", kI32, {E + 1}, dev);
    int64_t k = 1;
    const void *ids = nullptr;
    if (a[3] != Py_None) {
        k = whole(a[4]);
        if (k < 1 || k > 0x7fffffff) throw Refusal{PyExc_ValueError, "k must be at least 1"};
        ids = address(a[3], "sorted_ids", kI32, {M * k}, dev);
    }
    void *status = address(a[8], "status_out", kI32, {1}, dev, true);
    const at::Tensor out = output(a[6], "out", f32 ? kF32 : kBf16, {M * k, N}, dev);
    const int rc = moe_grouped_gemm(x.data_ptr(), wp, static_cast<const int32_t *>(offsets),
                                    static_cast<const int32_t *>(ids), out.data_ptr(), f32, swiglu, size(M), size(N),
                                    size(K), size(E), size(k), static_cast<int32_t *>(status), place.stream);
    if (rc != MOE_OK) return failed(rc, "moe_grouped_gemm");
    return THPVariable_Wrap(out);
    MOE_END
}

// (y, topk_w, inv_pos, add, out)
PyObject *combine(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    MOE_BEGIN("combine", 5)
    const bool f32 = tensor(a[0], "y").scalar_type() == kF32;
    const at::Tensor &y = lead(a[0], "y", f32 ? kF32 : kBf16);
    const at::Device dev = y.device();
    const Place place(dev);
    const at::Tensor &tw = tensor(a[1], "topk_w");
    const int64_t M = tw.dim() == 2 ? tw.size(0) : -1, k = tw.dim() == 2 ? tw.size(1) : -1, H = y.size(1);
    const void *w = address(a[1], "topk_w", kF32, {M, k}, dev);
    address(a[0], "y", f32 ? kF32 : kBf16, {M * k, H}, dev);
    const void *pos = address(a[2], "inv_pos", kI32, {M * k}, dev);
    const void *add = address(a[3], "add", kBf16, {M, H}, dev, true);
    const at::Tensor out = output(a[4], "out", kBf16, {M, H}, dev);
    const int rc = moe_combine(y.data_ptr(), f32, static_cast<const float *>(w), static_cast<const int32_t *>(pos), add,
                               out.data_ptr(), size(M), size(H), size(k), place.stream);
    if (rc != MOE_OK) return failed(rc, "moe_combine");
    return THPVariable_Wrap(out);
    MOE_END
}

#define MOE_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MOE_METHOD(block_norm), MOE_METHOD(int8_quantize), MOE_METHOD(int8_gemm),
                         MOE_METHOD(grouped_gemm), MOE_METHOD(combine),
                         {"raise_as", raise_as, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops(void) { return PyModule_Create(&module); }
