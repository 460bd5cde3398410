// ar_binding.cpp -- the marshalling of the paged key-value cache calls, as a
// CPython extension: checks of the tensors, allocation of results, and the
// call of the C ABI in libar.so (whose addresses bind() is given).  A decode
// step's kernels run for a few microseconds, and marshalling some forty sizes,
// strides and pointers a call by ctypes took three times as long.  Arguments
// are positional: the Python functions of the package name them.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <optional>
#include <string>

#include "ar.h"

namespace {

using at::Tensor;

decltype(&ar_kv_append) g_append = nullptr;
decltype(&ar_paged_attention_workspace_size) g_workspace_size = nullptr;
decltype(&ar_paged_attention) g_attention = nullptr;
decltype(&ar_attention_join) g_join = nullptr;
PyObject* g_error = nullptr;  // ARError

// Thrown with a Python exception set.
struct Raised {};

[[noreturn]] void bad(const std::string& what)
{
    PyErr_SetString(PyExc_ValueError, what.c_str());
    throw Raised();
}

void check(const char* func, int status)
{
    if (status == AR_OK)
        return;
    if (PyObject* e = PyObject_CallFunction(g_error, "si", func, status)) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised();
}

const Tensor& tensor(PyObject* o, const char* what)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
        throw Raised();
    }
    return THPVariable_Unpack(o);
}

bool given(PyObject* o) { return o != Py_None; }

double number(PyObject* o)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred())
        throw Raised();
    return x;
}

long long integer(PyObject* o)
{
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred())
        throw Raised();
    return x;
}

bool truth(PyObject* o)
{
    const int x = PyObject_IsTrue(o);
    if (x < 0)
        throw Raised();
    return x != 0;
}

int int32(PyObject* o, const char* what)
{
    const long long x = integer(o);
    if (x < INT32_MIN || x > INT32_MAX)
        bad(std::string(what) + " does not fit 32 bits");
    return static_cast<int>(x);
}

// A size of a tensor, as the C ABI's int.
int size32(int64_t n, const char* what)
{
    if (n > INT32_MAX)
        bad(std::string(what) + " has more rows than 32 bits count");
    return static_cast<int>(n);
}

int dtype_code(at::ScalarType t)
{
    switch (t) {
    case at::kFloat: return AR_FP32;
    case at::kHalf: return AR_FP16;
    case at::kBFloat16: return AR_BF16;
    default: bad(std::string("unsupported dtype ") + c10::toString(t) + "; expected float32, float16 or bfloat16");
    }
}

int cuda_index(const Tensor& t) { return t.is_cuda() ? static_cast<int>(t.get_device()) : -1; }

std::string on(int dev) { return " on cuda:" + std::to_string(dev); }

std::string shape_text(at::IntArrayRef s)
{
    std::string text = "[";
    for (size_t i = 0; i < s.size(); ++i)
        text += (i ? ", " : "") + std::to_string(s[i]);
    return text + "]";
}

// The stream of a call: an explicit handle, under which its results are then allocated too, so that the allocator hands
// out no memory that work queued elsewhere still uses; or the current one.
struct Stream {
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    ar_stream_t handle;
    Stream(PyObject* o, int dev)
    {
        if (given(o)) {
            const long long h = integer(o);
            handle = reinterpret_cast<ar_stream_t>(h);
            // 0 is the default stream, which torch knows by another name than an external one.
            guard.emplace(h == 0 ? c10::cuda::getDefaultCUDAStream(static_cast<c10::DeviceIndex>(dev))
                                 : c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(h), static_cast<c10::DeviceIndex>(dev)));
        } else {
            handle = reinterpret_cast<ar_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
        }
    }
};

// As torch.empty, without the way through the dispatcher.
Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& like)
{
    return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// Memory of the current stream's pool for one call: no tensor, and given back to that stream when the call is queued.
struct Scratch {
    void* p = nullptr;
    Scratch() = default;
    Scratch(const Scratch&) = delete;
    void make(size_t bytes) { p = c10::cuda::CUDACachingAllocator::raw_alloc(bytes); }
    ~Scratch()
    {
        if (p != nullptr)
            c10::cuda::CUDACachingAllocator::raw_delete(p);
    }
};

// A dense tensor of exactly this shape and type.
void dense(const Tensor& t, const char* what, at::IntArrayRef shape, at::ScalarType type, int dev)
{
    if (t.scalar_type() != type || t.sizes() != shape || cuda_index(t) != dev || !t.is_contiguous())
        bad(std::string(what) + " must be a contiguous " + c10::toString(type) + " tensor of shape " + shape_text(shape) + on(dev));
}

const int* ints(PyObject* o, const char* what, int64_t n, int dev)
{
    if (!given(o))
        return nullptr;
    const Tensor& t = tensor(o, what);
    dense(t, what, {n}, at::kInt, dev);
    return static_cast<const int*>(t.data_ptr());
}

// Elements between the rows of a [rows, heads, dim] tensor whose rows are dense; heads < 0: any number of them.
size_t row_stride(const Tensor& t, const char* what, int64_t rows, int64_t heads, int64_t dim, at::ScalarType type, int dev)
{
    if (t.dim() != 3 || t.size(0) != rows || (heads >= 0 && t.size(1) != heads) || t.size(2) != dim || t.scalar_type() != type ||
        cuda_index(t) != dev || (t.stride(2) != 1 && dim > 1) || (t.stride(1) != dim && t.size(1) > 1))
        bad(std::string(what) + " must be a [" + std::to_string(rows) + ", " + (heads < 0 ? "heads" : std::to_string(heads)) + ", " +
            std::to_string(dim) + "] " + c10::toString(type) + " tensor with dense rows" + on(dev));
    return static_cast<size_t>(t.stride(0));
}

// The cache's tensors, checked, and their device.
int fill_cache(ar_kv_cache* c, PyObject* k_pages, PyObject* v_pages, PyObject* page_table, PyObject* lengths, PyObject* layout,
               float k_scale, float v_scale)
{
    const Tensor& k = tensor(k_pages, "k_pages");
    const Tensor& v = tensor(v_pages, "v_pages");
    const Tensor& table = tensor(page_table, "page_table");
    int tokens = 0;
    if (PyUnicode_Check(layout) && PyUnicode_CompareWithASCIIString(layout, "NHD") == 0)
        tokens = 1;
    else if (PyUnicode_Check(layout) && PyUnicode_CompareWithASCIIString(layout, "HND") == 0)
        tokens = 2;
    else
        bad("layout must be 'NHD' ([pages, page_size, kv_heads, head_dim]) or 'HND' ([pages, kv_heads, page_size, head_dim])");
    const int heads = 3 - tokens, dev = cuda_index(k);
    if (dev < 0 || dev != c10::cuda::current_device())
        bad("k_pages must be a CUDA tensor of the current device");
    if (k.dim() != 4 || v.sizes() != k.sizes() || v.strides() != k.strides() || v.scalar_type() != k.scalar_type() ||
        cuda_index(v) != dev || (k.stride(3) != 1 && k.size(3) > 1))
        bad("k_pages and v_pages must be 4-d tensors of one shape, dtype, device and set of strides, with dense heads");
    const at::ScalarType type = k.scalar_type();
    if (type != at::kFloat && type != at::kHalf && type != at::kBFloat16 && type != at::kFloat8_e4m3fn)
        bad(std::string("unsupported cache dtype ") + c10::toString(type) + "; expected float32, float16, bfloat16 or float8_e4m3fn");
    if (table.dim() != 2 || table.scalar_type() != at::kInt || cuda_index(table) != dev || (table.stride(1) != 1 && table.size(1) > 1))
        bad("page_table must be an int32 [batch, pages of a sequence] tensor with dense rows" + on(dev));
    const int64_t batch = table.size(0), columns = table.size(1), stride = batch > 1 ? table.stride(0) : columns;
    if (stride < columns)
        bad("page_table's rows must not overlap");
    c->k = k.data_ptr();
    c->v = v.data_ptr();
    c->dtype = type == at::kFloat8_e4m3fn ? AR_FP8_E4M3 : dtype_code(type);
    c->pages = size32(k.size(0), "k_pages");
    c->page_size = size32(k.size(tokens), "k_pages");
    c->kv_heads = size32(k.size(heads), "k_pages");
    c->head_dim = size32(k.size(3), "k_pages");
    c->page_stride = static_cast<size_t>(k.stride(0));
    c->token_stride = static_cast<size_t>(k.stride(tokens));
    c->head_stride = static_cast<size_t>(k.stride(heads));
    c->k_scale = k_scale;
    c->v_scale = v_scale;
    c->page_table = static_cast<const int*>(table.data_ptr());
    c->batch = size32(batch, "page_table");
    c->max_pages = size32(columns, "page_table");
    c->table_stride = size32(stride, "page_table");
    if (!given(lengths))
        bad("lengths must be given");
    c->lengths = ints(lengths, "lengths", batch, dev);
    return dev;
}

// kv_append(k_pages, v_pages, page_table, lengths, k, v, q, q_out, seq_start, positions, inv_freq, interleaved,
//           rotary_scale, layout, k_scale, v_scale, stream)
PyObject* kv_append(PyObject* const* a)
{
    ar_kv_cache cache;
    const int dev = fill_cache(&cache, a[0], a[1], a[2], a[3], a[13], static_cast<float>(number(a[14])), static_cast<float>(number(a[15])));
    const Tensor& k = tensor(a[4], "k");
    const Tensor& v = tensor(a[5], "v");
    const at::ScalarType type = k.scalar_type();
    const int64_t tokens = k.dim() > 0 ? k.size(0) : 0, dim = cache.head_dim;
    ar_append_params p{};
    p.dtype = dtype_code(type);
    p.tokens = size32(tokens, "k");
    p.k_stride = row_stride(k, "k", tokens, cache.kv_heads, dim, type, dev);
    p.v_stride = row_stride(v, "v", tokens, cache.kv_heads, dim, type, dev);
    p.k = k.data_ptr();
    p.v = v.data_ptr();
    Stream s(a[16], dev);
    Tensor made;
    PyObject* result = Py_None;
    if (given(a[6])) {
        const Tensor& q = tensor(a[6], "q");
        p.q_stride = row_stride(q, "q", tokens, -1, dim, type, dev);
        p.q = q.data_ptr();
        p.q_heads = size32(q.size(1), "q");
        if (given(a[7])) {
            const Tensor& out = tensor(a[7], "q_out");
            p.q_out_stride = row_stride(out, "q_out", tokens, p.q_heads, dim, type, dev);
            p.q_out = out.data_ptr();
            result = a[7];
        } else {
            made = empty({tokens, p.q_heads, dim}, type, q);
            p.q_out_stride = static_cast<size_t>(p.q_heads) * dim;
            p.q_out = made.data_ptr();
        }
    } else if (given(a[7])) {
        bad("q_out is given without q");
    }
    p.seq_start = ints(a[8], "seq_start", static_cast<int64_t>(cache.batch) + 1, dev);
    p.positions = ints(a[9], "positions", tokens, dev);
    if (given(a[10])) {
        const Tensor& f = tensor(a[10], "inv_freq");
        if (f.scalar_type() != at::kFloat || cuda_index(f) != dev || !f.is_contiguous() || f.numel() > dim)
            bad("inv_freq must be a contiguous float32 tensor of at most head_dim / 2 elements" + on(dev));
        p.rotary_dim = static_cast<int>(2 * f.numel());
        p.inv_freq = static_cast<const float*>(f.data_ptr());
    }
    p.interleaved = truth(a[11]);
    p.rotary_scale = static_cast<float>(number(a[12]));
    check("ar_kv_append", g_append(&cache, &p, s.handle));
    if (made.defined())
        return THPVariable_Wrap(std::move(made));
    Py_INCREF(result);
    return result;
}

// paged_attention_workspace_size(k_pages, v_pages, page_table, lengths, q_heads, layout)
PyObject* paged_attention_workspace_size(PyObject* const* a)
{
    ar_kv_cache cache;
    fill_cache(&cache, a[0], a[1], a[2], a[3], a[5], 1.0f, 1.0f);
    return PyLong_FromSize_t(g_workspace_size(&cache, int32(a[4], "q_heads")));
}

// paged_attention(q, k_pages, v_pages, page_table, lengths, scale, window, softcap, layout, k_scale, v_scale, out, lse,
//                 return_lse, workspace, stream)
PyObject* paged_attention(PyObject* const* a)
{
    ar_kv_cache cache;
    const int dev = fill_cache(&cache, a[1], a[2], a[3], a[4], a[8], static_cast<float>(number(a[9])), static_cast<float>(number(a[10])));
    const Tensor& q = tensor(a[0], "q");
    const at::ScalarType type = q.scalar_type();
    const int code = dtype_code(type);
    const int64_t batch = cache.batch, dim = cache.head_dim;
    const size_t q_stride = row_stride(q, "q", batch, -1, dim, type, dev);
    const int q_heads = size32(q.size(1), "q");
    const float scale = given(a[5]) ? static_cast<float>(number(a[5])) : static_cast<float>(1.0 / std::sqrt(static_cast<double>(dim)));
    const int window = int32(a[6], "window");
    const float softcap = static_cast<float>(number(a[7]));
    Stream s(a[15], dev);
    Tensor out, lse;
    Scratch scratch;
    if (given(a[11])) {
        out = tensor(a[11], "out");
        dense(out, "out", {batch, q_heads, dim}, type, dev);
    } else {
        out = empty({batch, q_heads, dim}, type, q);
    }
    if (given(a[12])) {
        lse = tensor(a[12], "lse");
        dense(lse, "lse", {batch, q_heads}, at::kFloat, dev);
    } else if (truth(a[13])) {
        lse = empty({batch, q_heads}, at::kFloat, q);
    }
    void* workspace;
    size_t bytes;
    if (given(a[14])) {
        const Tensor& work = tensor(a[14], "workspace");
        if (cuda_index(work) != dev || !work.is_contiguous())
            bad("workspace must be a contiguous tensor" + on(dev));
        bytes = static_cast<size_t>(work.numel()) * work.element_size();
        workspace = work.data_ptr();
    } else {
        bytes = g_workspace_size(&cache, q_heads);
        if (bytes != 0)
            scratch.make(bytes);
        workspace = scratch.p;
    }
    check("ar_paged_attention",
          g_attention(&cache, q.data_ptr(), q_stride, q_heads, scale, window, softcap, out.data_ptr(),
                      lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, workspace, bytes, code, s.handle));
    if (!lse.defined())
        return THPVariable_Wrap(std::move(out));
    PyObject* x = THPVariable_Wrap(std::move(out));
    PyObject* y = x != nullptr ? THPVariable_Wrap(std::move(lse)) : nullptr;
    PyObject* both = y != nullptr ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return both;
}

// A list or tuple of at most AR_MAX_RANKS objects.
struct Items {
    PyObject* fast;
    Py_ssize_t n;
    Items(PyObject* o, const char* what) : fast(PySequence_Fast(o, what))
    {
        if (fast == nullptr)
            throw Raised();
        n = PySequence_Fast_GET_SIZE(fast);
    }
    ~Items() { Py_DECREF(fast); }
    Items(const Items&) = delete;
    PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

// attention_join(partials, lse, out, lse_out, return_lse, stream)
PyObject* attention_join(PyObject* const* a)
{
    const Items partials(a[0], "partials must be a sequence of tensors"), lses(a[1], "lse must be a sequence of tensors");
    if (partials.n == 0 || lses.n != partials.n)
        bad("ar_attention_join needs at least one partial, and one lse for each");
    if (partials.n > AR_MAX_RANKS)
        bad("ar_attention_join takes at most " + std::to_string(AR_MAX_RANKS) + " partials");
    const Tensor& p0 = tensor(partials[0], "partials[0]");
    const at::ScalarType type = p0.scalar_type();
    const int code = dtype_code(type), dev = cuda_index(p0);
    if (dev < 0 || dev != c10::cuda::current_device() || p0.dim() < 1)
        bad("partials must be [..., head_dim] CUDA tensors of the current device");
    const at::IntArrayRef shape = p0.sizes(), rows = shape.slice(0, shape.size() - 1);
    const void* x[AR_MAX_RANKS];
    const float* y[AR_MAX_RANKS];
    for (Py_ssize_t r = 0; r < partials.n; ++r) {
        const Tensor& p = tensor(partials[r], "partials");
        const Tensor& l = tensor(lses[r], "lse");
        dense(p, "every partial", shape, type, dev);
        dense(l, "every lse", rows, at::kFloat, dev);
        x[r] = p.data_ptr();
        y[r] = static_cast<const float*>(l.data_ptr());
    }
    Stream s(a[5], dev);
    Tensor out, lse;
    if (given(a[2])) {
        out = tensor(a[2], "out");
        dense(out, "out", shape, type, dev);
    } else {
        out = empty(shape, type, p0);
    }
    if (given(a[3])) {
        lse = tensor(a[3], "lse_out");
        dense(lse, "lse_out", rows, at::kFloat, dev);
    } else if (truth(a[4])) {
        lse = empty(rows, at::kFloat, p0);
    }
    const int64_t dim = shape.back();
    int64_t count = 1;
    for (int64_t n : rows)
        count *= n;
    check("ar_attention_join", g_join(x, y, static_cast<int>(partials.n), size32(count, "partials"), size32(dim, "partials"), out.data_ptr(),
                                      lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, code, s.handle));
    if (!lse.defined())
        return THPVariable_Wrap(std::move(out));
    PyObject* u = THPVariable_Wrap(std::move(out));
    PyObject* w = u != nullptr ? THPVariable_Wrap(std::move(lse)) : nullptr;
    PyObject* both = w != nullptr ? PyTuple_Pack(2, u, w) : nullptr;
    Py_XDECREF(u);
    Py_XDECREF(w);
    return both;
}

// bind(ARError, address of ar_kv_append, ..._workspace_size, ar_paged_attention, ar_attention_join)
PyObject* bind(PyObject* const* a)
{
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    g_append = reinterpret_cast<decltype(g_append)>(integer(a[1]));
    g_workspace_size = reinterpret_cast<decltype(g_workspace_size)>(integer(a[2]));
    g_attention = reinterpret_cast<decltype(g_attention)>(integer(a[3]));
    g_join = reinterpret_cast<decltype(g_join)>(integer(a[4]));
    Py_RETURN_NONE;
}

// Counts the arguments, and turns C++ exceptions into Python's.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    if (F != bind && g_error == nullptr) {
        PyErr_SetString(PyExc_RuntimeError, "the library is not loaded");
        return nullptr;
    }
    HANDLE_TH_ERRORS
    try {
        return F(args);
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int N>
constexpr PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<bind, 5>("bind"),
    method<kv_append, 17>("kv_append"),
    method<paged_attention_workspace_size, 6>("paged_attention_workspace_size"),
    method<paged_attention, 16>("paged_attention"),
    method<attention_join, 6>("attention_join"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
