// CPython binding of the attention side: bitlin_rope_apply, bitlin_kv_append and
// bitlin_kv_attend on torch tensors.  Argument checks and marshalling only; the
// calls are declared in include/bitlin.h and run in libbitlin.so.  It is compiled
// because these calls are small: marshalled through ctypes, one rotated token
// takes the host 9.7 us where the launch itself takes 2.
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <math.h>

#include "bitlin.h"

namespace {

// A Python error is set.
struct Refused {};

[[noreturn]] void refuse(const char* format, const char* what)
{
    PyErr_Format(PyExc_ValueError, format, what);
    throw Refused();
}

[[noreturn]] void refuse(const char* text)
{
    PyErr_SetString(PyExc_ValueError, text);
    throw Refused();
}

int cuda_error_of(bitlin_rope_t h) { return bitlin_rope_cuda_error(h); }
int cuda_error_of(bitlin_kv_t h) { return bitlin_kv_cuda_error(h); }

// Raises BitlinError for a call's status, with the CUDA error that the call left in its handle.
template <typename Handle>
void check(bitlin_status status, const char* call, Handle h)
{
    if (status == BITLIN_OK) return;
    const int cuda_error = status == BITLIN_ECUDA || status == BITLIN_ENOMEM ? cuda_error_of(h) : 0;
    PyObject* module = PyImport_ImportModule("hadamard_rotated_binary_gb300._binding");
    PyObject* type = module ? PyObject_GetAttrString(module, "BitlinError") : nullptr;
    PyObject* error = type ? PyObject_CallFunction(type, "isi", (int)status, call, cuda_error) : nullptr;
    if (error) PyErr_SetObject(type, error);
    Py_XDECREF(error);
    Py_XDECREF(type);
    Py_XDECREF(module);
    throw Refused();
}

void* handle_of(PyObject* o)
{
    void* h = o == Py_None ? nullptr : PyLong_AsVoidPtr(o);
    if (!h) {
        if (PyErr_Occurred()) throw Refused();
        refuse("the handle is closed");
    }
    return h;
}

long integer(PyObject* o)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}

const at::Tensor& tensor(PyObject* o, const char* what)
{
    if (!THPVariable_Check(o)) refuse("%s must be a torch tensor", what);
    return THPVariable_Unpack(o);
}

int type_of(at::ScalarType t)
{
    return t == at::kFloat ? BITLIN_F32 : t == at::kBFloat16 ? BITLIN_BF16 : t == at::kHalf ? BITLIN_F16 : -1;
}

// A kernel reads what it is given on the device of its handle alone.
void same_device(const at::Tensor& x, long device, const char* what)
{
    if (x.device().index() != device) refuse("%s must be on the handle's device", what);
}

// The C-ABI's view of a CUDA tensor [tokens][heads][dim] whose last dimension is contiguous.
bitlin_rows rows_of(const at::Tensor& x, long device, const char* what)
{
    const int type = type_of(x.scalar_type());
    if (type < 0 || !x.is_cuda() || x.dim() != 3)
        refuse("%s must be a float32, bfloat16 or float16 CUDA tensor [tokens][heads][dim]", what);
    same_device(x, device, what);
    if (x.stride(2) != 1 && x.size(2) != 1) refuse("%s's last dimension must be contiguous", what);
    // a dimension of one has no stride that matters
    const int64_t head = x.size(1) == 1 ? x.size(2) : x.stride(1);
    const int64_t token = x.size(0) == 1 ? x.size(1) * head : x.stride(0);
    return {x.data_ptr(), type, token, head};
}

// `out`, or a new tensor of x's shape and the given type.  A call on a stream of
// its own takes the new tensor's memory on that stream: the current one may still
// be using what its allocator would hand out, and the memory is not given out again
// before either stream is through with it.
at::Tensor output(PyObject* out, const at::Tensor& x, at::ScalarType type, PyObject* stream, bitlin_stream_t raw, const char* what)
{
    if (out == Py_None) {
        if (stream == Py_None) return at::empty(x.sizes(), x.options().dtype(type));
        const c10::DeviceIndex device = x.device().index();
        const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(device);
        at::Tensor t;
        {
            const c10::cuda::CUDAStreamGuard guard(
                c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(raw), device));
            t = at::empty(x.sizes(), x.options().dtype(type));
        }
        if (current.stream() != raw) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current);
        return t;
    }
    const at::Tensor& t = tensor(out, what);
    if (t.sizes() != x.sizes()) refuse("%s must have the input's shape", what);
    return t;
}

at::ScalarType dtype_of(PyObject* o, at::ScalarType otherwise)
{
    if (o == Py_None) return otherwise;
    if (!THPDtype_Check(o)) refuse("dtype must be a torch dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

bitlin_stream_t stream_of(PyObject* stream, const at::Tensor& x)
{
    if (stream == Py_None) return c10::cuda::getCurrentCUDAStream(x.device().index()).stream();
    PyObject* raw = PyObject_GetAttrString(stream, "cuda_stream");
    void* s = raw ? PyLong_AsVoidPtr(raw) : nullptr;
    Py_XDECREF(raw);
    if (PyErr_Occurred()) throw Refused();
    return static_cast<bitlin_stream_t>(s);
}

const int32_t* positions(PyObject* pos, long axes, int64_t tokens, long device)
{
    const at::Tensor& t = tensor(pos, "pos");
    if (t.scalar_type() != at::kInt || !t.is_cuda() || !t.is_contiguous() || t.numel() != axes * tokens)
        refuse("pos must be a contiguous int32 CUDA tensor [axes][tokens]");
    if (t.dim() > 1 && (t.dim() != 2 || t.size(0) != axes || t.size(1) != tokens))  // as many numbers in another order
        refuse("pos must be [axes][tokens]");
    same_device(t, device, "pos");
    return static_cast<const int32_t*>(t.data_ptr());
}

// Sizes reach the C-ABI as int.
int size_of(int64_t n)
{
    if (n > 0x7fffffff) refuse("too many tokens");
    return (int)n;
}

PyObject* wrap(const at::Tensor& t, PyObject* given)
{
    if (given == Py_None) return THPVariable_Wrap(t);
    Py_INCREF(given);
    return given;
}

bool arguments(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
    return n == want;
}

// (handle, device, axes, x, pos, out, dtype, inverse, stream)
PyObject* rope_apply(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!arguments(n, 9)) return nullptr;
    HANDLE_TH_ERRORS
    try {
        auto h = static_cast<bitlin_rope_t>(handle_of(a[0]));
        const long device = integer(a[1]);
        const at::Tensor& x = tensor(a[3], "x");
        const bitlin_rows src = rows_of(x, device, "x");
        const int32_t* pos = positions(a[4], integer(a[2]), x.size(0), device);
        const bitlin_stream_t stream = stream_of(a[8], x);
        const at::Tensor out = output(a[5], x, dtype_of(a[6], x.scalar_type()), a[8], stream, "out");
        const bitlin_rows dst = rows_of(out, device, "out");
        check(bitlin_rope_apply(h, &src, size_of(x.size(0)), size_of(x.size(1)), size_of(x.size(2)), pos, &dst,
                                PyObject_IsTrue(a[7]), stream),
              "bitlin_rope_apply", h);
        return wrap(out, a[5]);
    } catch (const Refused&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (handle, device, kv_heads, head_dim, cache dtype, batch, k, v, rope, axes, pos, q, q_out, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!arguments(n, 14)) return nullptr;
    HANDLE_TH_ERRORS
    try {
        auto h = static_cast<bitlin_kv_t>(handle_of(a[0]));
        const long device = integer(a[1]);
        const long kv_heads = integer(a[2]), dim = integer(a[3]);
        const at::ScalarType type = dtype_of(a[4], at::kFloat);
        const auto* batch = static_cast<const bitlin_kv_batch*>(handle_of(a[5]));
        const at::Tensor &k = tensor(a[6], "k"), &v = tensor(a[7], "v");
        const bitlin_rows kr = rows_of(k, device, "k"), vr = rows_of(v, device, "v");
        if (k.sizes() != v.sizes() || k.size(1) != kv_heads || k.size(2) != dim)
            refuse("k and v must be [tokens][kv_heads][head_dim]");
        const int64_t tokens = k.size(0);
        const bitlin_stream_t stream = stream_of(a[13], k);
        bitlin_rope_t rope = nullptr;
        const int32_t* pos = nullptr;
        if (a[8] != Py_None) {
            rope = static_cast<bitlin_rope_t>(handle_of(a[8]));
            if (a[10] != Py_None) pos = positions(a[10], integer(a[9]), tokens, device);
        }
        bitlin_rows qr = {}, or_ = {};
        at::Tensor out;
        int heads = 0;
        if (a[11] != Py_None) {
            const at::Tensor& q = tensor(a[11], "q");
            qr = rows_of(q, device, "q");
            if (q.size(0) != tokens || q.size(2) != dim) refuse("q must be [tokens][heads][head_dim]");
            heads = size_of(q.size(1));
            out = output(a[12], q, type, a[13], stream, "q_out");
            or_ = rows_of(out, device, "q_out");
        }
        const bool has_q = a[11] != Py_None;
        check(bitlin_kv_append(h, batch, size_of(tokens), rope, pos, &kr, &vr, has_q ? &qr : nullptr, heads,
                               has_q ? &or_ : nullptr, stream),
              "bitlin_kv_append", h);
        if (has_q) return wrap(out, a[12]);
        Py_RETURN_NONE;
    } catch (const Refused&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (handle, device, head_dim, cache dtype, batch, q, scale, causal, out, dtype, lse, stream)
PyObject* kv_attend(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (!arguments(n, 12)) return nullptr;
    HANDLE_TH_ERRORS
    try {
        auto h = static_cast<bitlin_kv_t>(handle_of(a[0]));
        const long device = integer(a[1]);
        const long dim = integer(a[2]);
        const at::ScalarType type = dtype_of(a[3], at::kFloat);
        const auto* batch = static_cast<const bitlin_kv_batch*>(handle_of(a[4]));
        const at::Tensor& q = tensor(a[5], "q");
        const bitlin_rows qr = rows_of(q, device, "q");
        if (q.size(2) != dim) refuse("q must be [tokens][heads][head_dim]");
        double scale = 1.0 / sqrt((double)dim);
        if (a[6] != Py_None) {
            scale = PyFloat_AsDouble(a[6]);
            if (scale == -1.0 && PyErr_Occurred()) throw Refused();
        }
        const bitlin_stream_t stream = stream_of(a[11], q);
        const at::Tensor out = output(a[8], q, dtype_of(a[9], type), a[11], stream, "out");
        const bitlin_rows dst = rows_of(out, device, "out");
        float* lse = nullptr;
        if (a[10] != Py_None) {
            const at::Tensor& t = tensor(a[10], "lse");
            if (t.scalar_type() != at::kFloat || !t.is_cuda() || !t.is_contiguous() || t.dim() != 2 ||
                t.size(0) != q.size(0) || t.size(1) != q.size(1))
                refuse("lse must be a contiguous float32 CUDA tensor [tokens][heads]");
            same_device(t, device, "lse");
            lse = static_cast<float*>(t.data_ptr());
        }
        check(bitlin_kv_attend(h, batch, size_of(q.size(0)), &qr, size_of(q.size(1)), (float)scale,
                               PyObject_IsTrue(a[7]), &dst, lse, stream),
              "bitlin_kv_attend", h);
        return wrap(out, a[8]);
    } catch (const Refused&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL

PyMethodDef methods[] = {
    {"rope_apply", FAST(rope_apply), nullptr},
    {"kv_append", FAST(kv_append), nullptr},
    {"kv_attend", FAST(kv_attend), nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_native(void) { return PyModule_Create(&module); }
