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
decltype(&ar_kv_append_axes) g_append_axes = nullptr;
decltype(&ar_kv_compact) g_compact = nullptr;
decltype(&ar_kv_copy_pages) g_copy_pages = nullptr;
decltype(&ar_tree_attention_workspace_size) g_tree_workspace_size = nullptr;
decltype(&ar_tree_attention) g_tree = nullptr;
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

// Which dimension of the pages counts tokens.
int token_dim(PyObject* layout)
{
    if (PyUnicode_Check(layout) && PyUnicode_CompareWithASCIIString(layout, "NHD") == 0)
        return 1;
    if (PyUnicode_Check(layout) && PyUnicode_CompareWithASCIIString(layout, "HND") == 0)
        return 2;
    bad("layout must be 'NHD' ([pages, page_size, kv_heads, head_dim]) or 'HND' ([pages, kv_heads, page_size, head_dim])");
}

// The pages' tensors, checked, and their device.  tokens: the dimension that counts them; 0 where the call takes either for it:
// then the longer one, as heads are 1024 at the most and a page's tokens any number.
int fill_pages(ar_kv_cache* c, const Tensor& k, const Tensor& v, int tokens)
{
    const int dev = cuda_index(k);
    if (dev < 0 || dev != c10::cuda::current_device())
        bad("k_pages must be a CUDA tensor of the current device");
    if (k.dim() != 4 || v.sizes() != k.sizes() || v.strides() != k.strides() || v.scalar_type() != k.scalar_type() ||
        cuda_index(v) != dev || (k.stride(3) != 1 && k.size(3) > 1))
        bad("k_pages and v_pages must be 4-d tensors of one shape, dtype, device and set of strides, with dense heads");
    if (tokens == 0)
        tokens = k.sizes()[2] > k.sizes()[1] ? 2 : 1;
    const int heads = 3 - tokens;
    const at::ScalarType type = k.scalar_type();
    if (type != at::kFloat && type != at::kHalf && type != at::kBFloat16 && type != at::kFloat8_e4m3fn)
        bad(std::string("unsupported cache dtype ") + c10::toString(type) + "; expected float32, float16, bfloat16 or float8_e4m3fn");
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
    return dev;
}

// The page table and the lengths.
void fill_table(ar_kv_cache* c, PyObject* page_table, PyObject* lengths, int dev)
{
    const Tensor& table = tensor(page_table, "page_table");
    if (table.dim() != 2 || table.scalar_type() != at::kInt || cuda_index(table) != dev || (table.stride(1) != 1 && table.size(1) > 1))
        bad("page_table must be an int32 [batch, pages of a sequence] tensor with dense rows" + on(dev));
    const int64_t batch = table.size(0), columns = table.size(1), stride = batch > 1 ? table.stride(0) : columns;
    if (stride < columns)
        bad("page_table's rows must not overlap");
    c->page_table = static_cast<const int*>(table.data_ptr());
    c->batch = size32(batch, "page_table");
    c->max_pages = size32(columns, "page_table");
    c->table_stride = size32(stride, "page_table");
    if (!given(lengths))
        bad("lengths must be given");
    c->lengths = ints(lengths, "lengths", batch, dev);
}

// The cache's tensors, checked, and their device.
int fill_cache(ar_kv_cache* c, PyObject* k_pages, PyObject* v_pages, PyObject* page_table, PyObject* lengths, PyObject* layout,
               float k_scale, float v_scale)
{
    const int tokens = token_dim(layout);
    const int dev = fill_pages(c, tensor(k_pages, "k_pages"), tensor(v_pages, "v_pages"), tokens);
    fill_table(c, page_table, lengths, dev);
    c->k_scale = k_scale;
    c->v_scale = v_scale;
    return dev;
}

// A list or tuple of objects.
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

// The pages of several layers, one tensor or a sequence of them each, of one shape.
struct LayerPages {
    void* k[AR_MAX_LAYERS];
    void* v[AR_MAX_LAYERS];
    int n, dev;
    LayerPages(ar_kv_cache* c, PyObject* k_pages, PyObject* v_pages, int tokens)
    {
        if (THPVariable_Check(k_pages) && THPVariable_Check(v_pages)) {
            n = 1;
            dev = fill_pages(c, THPVariable_Unpack(k_pages), THPVariable_Unpack(v_pages), tokens);
            k[0] = c->k;
            v[0] = c->v;
            return;
        }
        const Items ks(k_pages, "k_pages must be a tensor or a sequence of tensors"), vs(v_pages, "v_pages must be a tensor or a sequence of tensors");
        if (ks.n < 1 || ks.n != vs.n || ks.n > AR_MAX_LAYERS)
            bad("k_pages and v_pages must name the same layers, 1 to " + std::to_string(AR_MAX_LAYERS));
        n = static_cast<int>(ks.n);
        for (int i = 0; i < n; ++i) {
            const Tensor& x = tensor(ks[i], "k_pages");
            const Tensor& y = tensor(vs[i], "v_pages");
            const Tensor& first = tensor(ks[0], "k_pages");
            if (x.sizes() != first.sizes() || x.strides() != first.strides() || x.scalar_type() != first.scalar_type())
                bad("all layers' pages must have one shape, dtype and set of strides");
            dev = fill_pages(c, x, y, tokens);
            k[i] = c->k;
            v[i] = c->v;
        }
    }
};

// kv_append(k_pages, v_pages, page_table, lengths, k, v, q, q_out, seq_start, positions, inv_freq, interleaved,
//           rotary_scale, layout, k_scale, v_scale, stream, pair_axis)
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
    unsigned char pair_axis[512];
    int axes = 0;
    size_t axis_stride = 0;
    Py_ssize_t pairs = 0;
    if (given(a[17])) {
        const Items axis(a[17], "pair_axis must be a sequence of whole numbers");
        const Tensor& x = tensor(a[9], "positions");
        if (x.dim() != 2 || x.size(0) < 1 || x.size(0) > AR_MAX_AXES || x.size(1) != tokens || x.scalar_type() != at::kInt || cuda_index(x) != dev ||
            (x.stride(1) != 1 && tokens > 1) || (x.size(0) > 1 && x.stride(0) < tokens))
            bad("positions must be an int32 [axes, " + std::to_string(tokens) + "] tensor with dense rows, 1 to " + std::to_string(AR_MAX_AXES) +
                " of them" + on(dev));
        axes = static_cast<int>(x.size(0));
        axis_stride = static_cast<size_t>(x.stride(0));
        p.positions = static_cast<const int*>(x.data_ptr());
        pairs = axis.n;
        if (pairs > 512)
            bad("pair_axis must have one entry for each element of inv_freq");
        for (Py_ssize_t j = 0; j < pairs; ++j) {
            const long long x = integer(axis[j]);
            if (x < 0 || x >= axes)
                bad("pair_axis must hold numbers from 0 to " + std::to_string(axes - 1));
            pair_axis[j] = static_cast<unsigned char>(x);
        }
    } else {
        p.positions = ints(a[9], "positions", tokens, dev);
    }
    if (given(a[10])) {
        const Tensor& f = tensor(a[10], "inv_freq");
        if (f.scalar_type() != at::kFloat || cuda_index(f) != dev || !f.is_contiguous() || f.numel() > dim)
            bad("inv_freq must be a contiguous float32 tensor of at most head_dim / 2 elements" + on(dev));
        p.rotary_dim = static_cast<int>(2 * f.numel());
        p.inv_freq = static_cast<const float*>(f.data_ptr());
    }
    p.interleaved = truth(a[11]);
    p.rotary_scale = static_cast<float>(number(a[12]));
    if (axes > 0) {
        if (2 * pairs != p.rotary_dim)
            bad("pair_axis must have one entry for each element of inv_freq");
        check("ar_kv_append_axes", g_append_axes(&cache, &p, axes, axis_stride, pair_axis, s.handle));
    } else {
        check("ar_kv_append", g_append(&cache, &p, s.handle));
    }
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

// kv_compact(k_pages, v_pages, page_table, lengths, kept, seq_start, drafted, layout, new_lengths, stream)
PyObject* kv_compact(PyObject* const* a)
{
    ar_kv_cache cache{};
    const LayerPages layers(&cache, a[0], a[1], token_dim(a[7]));
    const int dev = layers.dev;
    fill_table(&cache, a[2], a[3], dev);
    const Tensor& kept = tensor(a[4], "kept");
    if (kept.dim() != 2 || kept.size(0) != cache.batch || kept.scalar_type() != at::kInt || cuda_index(kept) != dev ||
        (kept.stride(1) != 1 && kept.size(1) > 1) || (cache.batch > 1 && kept.stride(0) < kept.size(1)))
        bad("kept must be an int32 [batch, kept tokens] tensor with dense rows" + on(dev));
    const int* seq_start = ints(a[5], "seq_start", static_cast<int64_t>(cache.batch) + 1, dev);
    if ((seq_start != nullptr) == given(a[6]))
        bad("either seq_start or drafted must be given");
    const int drafted = given(a[6]) ? int32(a[6], "drafted") : 0;
    Stream s(a[9], dev);
    Tensor out;
    if (given(a[8])) {
        out = tensor(a[8], "new_lengths");
        dense(out, "new_lengths", {cache.batch}, at::kInt, dev);
    } else {
        out = empty({cache.batch}, at::kInt, kept);
    }
    check("ar_kv_compact", g_compact(&cache, layers.k, layers.v, layers.n, static_cast<const int*>(kept.data_ptr()), static_cast<size_t>(kept.stride(0)),
                                     size32(kept.size(1), "kept"), seq_start, drafted, static_cast<int*>(out.data_ptr()), s.handle));
    return THPVariable_Wrap(std::move(out));
}

// kv_copy_pages(k_pages, v_pages, src, dst, stream)
PyObject* kv_copy_pages(PyObject* const* a)
{
    ar_kv_cache cache{};
    const LayerPages layers(&cache, a[0], a[1], 0);  // whole pages: which dimension counts tokens does not matter
    const int dev = layers.dev;
    const Tensor& src = tensor(a[2], "src");
    const Tensor& dst = tensor(a[3], "dst");
    if (src.dim() != 1)
        bad("src must be an int32 [pairs] tensor" + on(dev));
    dense(src, "src", {src.size(0)}, at::kInt, dev);
    dense(dst, "dst", {src.size(0)}, at::kInt, dev);
    Stream s(a[4], dev);
    check("ar_kv_copy_pages", g_copy_pages(&cache, layers.k, layers.v, layers.n, static_cast<const int*>(src.data_ptr()),
                                           static_cast<const int*>(dst.data_ptr()), size32(src.size(0), "src"), s.handle));
    Py_RETURN_NONE;
}

// tree_attention_workspace_size(k_pages, v_pages, page_table, lengths, q_heads, tokens, layout)
PyObject* tree_attention_workspace_size(PyObject* const* a)
{
    ar_kv_cache cache;
    fill_cache(&cache, a[0], a[1], a[2], a[3], a[6], 1.0f, 1.0f);
    return PyLong_FromSize_t(g_tree_workspace_size(&cache, int32(a[4], "q_heads"), int32(a[5], "tokens")));
}

// tree_attention(q, k_pages, v_pages, page_table, lengths, mask, seq_start, scale, window, softcap, layout, k_scale, v_scale,
//                out, lse, return_lse, workspace, stream)
PyObject* tree_attention(PyObject* const* a)
{
    ar_kv_cache cache;
    const int dev = fill_cache(&cache, a[1], a[2], a[3], a[4], a[10], static_cast<float>(number(a[11])), static_cast<float>(number(a[12])));
    const Tensor& q = tensor(a[0], "q");
    const at::ScalarType type = q.scalar_type();
    const int64_t tokens = q.dim() > 0 ? q.size(0) : 0, dim = cache.head_dim;
    ar_tree_params p{};
    p.dtype = dtype_code(type);
    p.tokens = size32(tokens, "q");
    p.q_stride = row_stride(q, "q", tokens, -1, dim, type, dev);
    p.q = q.data_ptr();
    p.q_heads = size32(q.size(1), "q");
    if (given(a[5])) {
        const Tensor& mask = tensor(a[5], "mask");
        if (mask.dim() != 2)
            bad("mask must be an int64 [" + std::to_string(tokens) + ", words] tensor" + on(dev));
        dense(mask, "mask", {tokens, mask.size(1)}, at::kLong, dev);
        p.mask_words = size32(mask.size(1), "mask");
        if (p.mask_words < 1)
            bad("mask must have one word of 64 tokens at least");
        p.mask = static_cast<const uint64_t*>(mask.data_ptr());
    }
    p.seq_start = ints(a[6], "seq_start", static_cast<int64_t>(cache.batch) + 1, dev);
    p.scale = given(a[7]) ? static_cast<float>(number(a[7])) : static_cast<float>(1.0 / std::sqrt(static_cast<double>(dim)));
    p.window = int32(a[8], "window");
    p.softcap = static_cast<float>(number(a[9]));
    Stream s(a[17], dev);
    Tensor out, lse;
    Scratch scratch;
    if (given(a[13])) {
        out = tensor(a[13], "out");
        dense(out, "out", {tokens, p.q_heads, dim}, type, dev);
    } else {
        out = empty({tokens, p.q_heads, dim}, type, q);
    }
    if (given(a[14])) {
        lse = tensor(a[14], "lse");
        dense(lse, "lse", {tokens, p.q_heads}, at::kFloat, dev);
    } else if (truth(a[15])) {
        lse = empty({tokens, p.q_heads}, at::kFloat, q);
    }
    p.out = out.data_ptr();
    p.lse = lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr;
    void* workspace;
    size_t bytes;
    if (given(a[16])) {
        const Tensor& work = tensor(a[16], "workspace");
        if (cuda_index(work) != dev || !work.is_contiguous())
            bad("workspace must be a contiguous tensor" + on(dev));
        bytes = static_cast<size_t>(work.numel()) * work.element_size();
        workspace = work.data_ptr();
    } else {
        bytes = g_tree_workspace_size(&cache, p.q_heads, p.tokens);
        if (bytes != 0)
            scratch.make(bytes);
        workspace = scratch.p;
    }
    check("ar_tree_attention", g_tree(&cache, &p, workspace, bytes, s.handle));
    if (!lse.defined())
        return THPVariable_Wrap(std::move(out));
    PyObject* x = THPVariable_Wrap(std::move(out));
    PyObject* y = x != nullptr ? THPVariable_Wrap(std::move(lse)) : nullptr;
    PyObject* both = y != nullptr ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return both;
}

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

// bind(ARError, address of ar_kv_append, ar_paged_attention_workspace_size, ar_paged_attention, ar_attention_join,
//      ar_kv_append_axes, ar_kv_compact, ar_kv_copy_pages, ar_tree_attention_workspace_size, ar_tree_attention)
PyObject* bind(PyObject* const* a)
{
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    g_append = reinterpret_cast<decltype(g_append)>(integer(a[1]));
    g_workspace_size = reinterpret_cast<decltype(g_workspace_size)>(integer(a[2]));
    g_attention = reinterpret_cast<decltype(g_attention)>(integer(a[3]));
    g_join = reinterpret_cast<decltype(g_join)>(integer(a[4]));
    g_append_axes = reinterpret_cast<decltype(g_append_axes)>(integer(a[5]));
    g_compact = reinterpret_cast<decltype(g_compact)>(integer(a[6]));
    g_copy_pages = reinterpret_cast<decltype(g_copy_pages)>(integer(a[7]));
    g_tree_workspace_size = reinterpret_cast<decltype(g_tree_workspace_size)>(integer(a[8]));
    g_tree = reinterpret_cast<decltype(g_tree)>(integer(a[9]));
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
    method<bind, 10>("bind"),
    method<kv_append, 18>("kv_append"),
    method<paged_attention_workspace_size, 6>("paged_attention_workspace_size"),
    method<paged_attention, 16>("paged_attention"),
    method<attention_join, 6>("attention_join"),
    method<kv_compact, 10>("kv_compact"),
    method<kv_copy_pages, 5>("kv_copy_pages"),
    method<tree_attention_workspace_size, 7>("tree_attention_workspace_size"),
    method<tree_attention, 18>("tree_attention"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
