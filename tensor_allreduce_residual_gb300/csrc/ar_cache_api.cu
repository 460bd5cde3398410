// ar_cache_api.cu -- the C ABI of the paged key-value cache calls: argument
// checks, launch shapes and dispatch on the element types.  Host code only; it
// allocates nothing.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <initializer_list>

#include "ar.h"
#include "ar_cache.h"
#include "ar_tree.h"

namespace {

constexpr int kMaxHeads = 1024;
constexpr int kMaxHeadDim = 1024;

int esize_of(int dtype) { return dtype == AR_FP32 ? 4 : dtype == AR_FP16 || dtype == AR_BF16 ? 2 : 0; }

int cache_esize_of(int dtype) { return dtype == AR_FP8_E4M3 ? 1 : esize_of(dtype); }

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

int status_of(cudaError_t e) { return e == cudaSuccess ? AR_OK : AR_ERR_CUDA; }

bool scale_ok(float s) { return std::isfinite(s) && s > 0.0f; }

// The cache with the strides that no element needs (one page, token or head) set to 0, so that they refuse nothing.
ar_kv_cache without_idle_strides(const ar_kv_cache* cache)
{
    ar_kv_cache c{};
    if (cache != nullptr)
        c = *cache;
    c.page_stride = c.pages > 1 ? c.page_stride : 0;
    c.token_stride = c.page_size > 1 ? c.token_stride : 0;
    c.head_stride = c.kv_heads > 1 ? c.head_stride : 0;
    return c;
}

// Sizes and strides of the pages (all zeros for a NULL cache); no pointer is looked at.
bool page_sizes_ok(const ar_kv_cache* c)
{
    return c->pages >= 1 && c->page_size >= 1 && c->kv_heads >= 1 && c->head_dim >= 1;
}
bool table_ok(const ar_kv_cache* c) { return c->batch >= 0 && c->max_pages >= 1 && c->table_stride >= c->max_pages; }
bool page_limits_ok(const ar_kv_cache* c)
{
    return cache_esize_of(c->dtype) != 0 && c->kv_heads <= kMaxHeads && c->head_dim <= kMaxHeadDim;
}
bool page_strides_ok(const ar_kv_cache* c)
{
    const size_t d = static_cast<size_t>(c->head_dim);
    return (c->pages == 1 || c->page_stride >= d) && (c->page_size == 1 || c->token_stride >= d) &&
           (c->kv_heads == 1 || c->head_stride >= d);
}

// Sizes, strides and dtype of the cache (all zeros for a NULL one); no pointer is looked at.
int check_sizes(const ar_kv_cache* c)
{
    if (!page_sizes_ok(c) || !table_ok(c))
        return AR_ERR_INVALID_ARG;
    if (!page_limits_ok(c))
        return AR_ERR_UNSUPPORTED;
    if (!page_strides_ok(c) || !scale_ok(c->k_scale) || !scale_ok(c->v_scale))
        return AR_ERR_INVALID_ARG;
    return AR_OK;
}

// The caches of several layers: their shared shape (with its table where `table`), and how many they are.
int check_layers(const ar_kv_cache* c, int layers, bool table)
{
    if (!page_sizes_ok(c) || (table && !table_ok(c)) || layers < 1)
        return AR_ERR_INVALID_ARG;
    if (!page_limits_ok(c) || layers > AR_MAX_LAYERS)
        return AR_ERR_UNSUPPORTED;
    return page_strides_ok(c) ? AR_OK : AR_ERR_INVALID_ARG;
}

int check_dtypes(int dtype, int cache_dtype)
{
    if (esize_of(dtype) == 0 || !(cache_dtype == dtype || (cache_dtype == AR_FP8_E4M3 && dtype != AR_FP32)))
        return AR_ERR_UNSUPPORTED;
    return AR_OK;
}

bool element_ok(const void* p, size_t esize) { return p != nullptr && aligned(p, esize); }

bool pointers_ok(const ar_kv_cache* c)
{
    const size_t e = static_cast<size_t>(cache_esize_of(c->dtype));
    return element_ok(c->k, e) && element_ok(c->v, e) && element_ok(c->page_table, 4) && element_ok(c->lengths, 4);
}

// Calls f(T{}, CT{}) with the element types of the tensors and of the cache.
template <typename F>
cudaError_t by_dtypes(int dtype, int cache_dtype, F&& f)
{
    const bool small = cache_dtype == AR_FP8_E4M3;
    switch (dtype) {
    case AR_FP32: return f(float{}, float{});
    case AR_FP16: return small ? f(__half{}, __nv_fp8_e4m3{}) : f(__half{}, __half{});
    default: return small ? f(__nv_bfloat16{}, __nv_fp8_e4m3{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
    }
}

uint64_t magic_of(int units) { return ((1ull << 32) + units - 1) / units; }

// Sizes of ar_paged_attention that both it and its workspace size check.
int check_attention(const ar_kv_cache* c, int q_heads)
{
    if (int st = check_sizes(c))
        return st;
    if (q_heads < 1 || q_heads % c->kv_heads != 0)
        return AR_ERR_INVALID_ARG;
    const size_t e = static_cast<size_t>(cache_esize_of(c->dtype));
    if (q_heads > kMaxHeads || c->head_dim > ar::kAttnMaxDim || c->head_dim * e % 16 != 0 ||
        c->page_stride * e % 16 != 0 || c->token_stride * e % 16 != 0 || c->head_stride * e % 16 != 0)
        return AR_ERR_UNSUPPORTED;
    return AR_OK;
}

int group_blocks_of(const ar_kv_cache* c, int q_heads)
{
    const int block_heads = ar::attn_block_heads(cache_esize_of(c->dtype));
    return (q_heads / c->kv_heads + block_heads - 1) / block_heads;
}

// Sequences times key-value heads times blocks of query heads.
size_t attention_items(const ar_kv_cache* c, int q_heads)
{
    return static_cast<size_t>(c->batch) * c->kv_heads * group_blocks_of(c, q_heads);
}

int slot_floats_of(const ar_kv_cache* c, int q_heads)
{
    const int group = q_heads / c->kv_heads, block_heads = ar::attn_block_heads(cache_esize_of(c->dtype));
    return ar::attn_slot_floats(group < block_heads ? group : block_heads, c->head_dim);
}

// Blocks of the attention kernel, at most: no more than there can be tiles.
int attention_blocks(const ar_kv_cache* c, int q_heads)
{
    const long long cap = static_cast<long long>(c->max_pages) * c->page_size;
    const long long tile = ar::attn_tile(cache_esize_of(c->dtype), c->head_dim);
    const long long items = static_cast<long long>(attention_items(c, q_heads));
    const long long tiles = (cap < INT_MAX ? cap : INT_MAX) / tile + 2;
    const long long most = ar::kAttnMaxBlocks;
    return static_cast<int>(items >= most || items * tiles >= most ? most : items * tiles);
}

// token / page_size == (2 token * magic >> 32) >> shift for token < 2^31: m = ceil(2^(31 + l) / d) with 2^l the power of two
// from d on is below 2^32, and n m >> (31 + l) = n / d below 2^31.
void page_division(int page_size, uint32_t* magic, int* shift)
{
    *shift = 0;
    while ((1ll << *shift) < page_size)
        ++*shift;
    *magic = static_cast<uint32_t>(((1ull << (31 + *shift)) + page_size - 1) / page_size);
}

// Tokens that a row of the table can hold; a tile's end stays an int.
int capacity_of(const ar_kv_cache* c)
{
    const long long cap = static_cast<long long>(c->max_pages) * c->page_size;
    return static_cast<int>(cap < INT_MAX - 255 ? cap : INT_MAX - 255);
}

// The factors of scores in base 2: false where one is not finite, which would make scores of 0 NaN.
bool score_factors(float scale, float k_scale, float softcap, float* scale2, float* softcap2)
{
    constexpr float kLog2e = 1.4426950408889634f;
    *scale2 = scale * k_scale * kLog2e * (softcap > 0.0f ? 2.0f / softcap : 1.0f);
    *softcap2 = softcap * kLog2e;
    return std::isfinite(*scale2) && std::isfinite(*softcap2);
}

// Sizes of ar_tree_attention that both it and its workspace size check.
int check_tree(const ar_kv_cache* c, int q_heads, int tokens)
{
    if (int st = check_attention(c, q_heads))
        return st;
    if (tokens < 0)
        return AR_ERR_INVALID_ARG;
    return static_cast<uint64_t>(tokens) * (q_heads / c->kv_heads) <= INT_MAX - 255 ? AR_OK : AR_ERR_UNSUPPORTED;
}

// The driver's encoder of tensor maps, or nullptr.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static std::atomic<void*> found{nullptr};
    void* f = found.load(std::memory_order_acquire);
    if (f == nullptr) {
        cudaDriverEntryPointQueryResult how;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &how) != cudaSuccess ||
            how != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        found.store(f, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

// Describes the pages for tensor copies, where they can be: pages of whole groups of eight tokens.  Returns a copy's tokens, the
// largest power of two that divides a page, `tile` at most; 0: they cannot be.  16-bit elements come by 64, 8-bit ones by `dim`.
int tree_maps(const ar_kv_cache* c, int tile, int dim, ar::TreeMaps* maps, int* token_first)
{
    const uint64_t e = static_cast<uint64_t>(cache_esize_of(c->dtype));
    const int whole = c->page_size & -c->page_size, tokens = whole < tile ? whole : tile;
    if (e == 4 || tokens < 8)
        return 0;
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr)
        return 0;
    // An axis of one element needs no stride, but an allowed one.
    const uint64_t page = c->page_stride * e, token = c->token_stride * e, head = c->head_stride * e;
    const auto some = [](uint64_t stride) { return stride != 0 ? stride : 16; };
    *token_first = c->kv_heads == 1 || token <= head;
    const cuuint64_t sizes[4] = {static_cast<cuuint64_t>(c->head_dim), static_cast<cuuint64_t>(*token_first ? c->page_size : c->kv_heads),
                                 static_cast<cuuint64_t>(*token_first ? c->kv_heads : c->page_size), static_cast<cuuint64_t>(c->pages)};
    const cuuint64_t strides[3] = {some(*token_first ? token : head), some(*token_first ? head : token), some(page)};
    const cuuint32_t rows = static_cast<cuuint32_t>(tokens);
    const cuuint32_t box[4] = {e == 1 ? static_cast<cuuint32_t>(dim) : 64u, *token_first ? rows : 1u, *token_first ? 1u : rows, 1u};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = e == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                            : c->dtype == AR_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const auto map = [&](CUtensorMap* to, void* pages) {
        return encode(to, type, 4, pages, sizes, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      e == 1 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    return map(&maps->k, c->k) && map(&maps->v, c->v) ? tokens : 0;
}

// Fault injection of the tests: the test build of the library (compiled with AR_TEST_HOOKS, libar_test.so) reads it once from
// AR_TEST_TREE_STALL; the product library never reads the environment.
int tree_stall()
{
#ifdef AR_TEST_HOOKS
    static const int stall = [] {
        const char* e = std::getenv("AR_TEST_TREE_STALL");
        return e != nullptr ? std::atoi(e) : 0;
    }();
    return stall;
#else
    return 0;
#endif
}

struct TreePlan {
    ar::TreeShape shape;
    int blocks, slot_rows;
    size_t slot_floats, part_at, bytes;
};

TreePlan tree_plan(const ar_kv_cache* c, int q_heads, int tokens)
{
    TreePlan p{};
    const uint64_t rows = static_cast<uint64_t>(tokens) * (q_heads / c->kv_heads);
    p.shape = ar::tree_shape(cache_esize_of(c->dtype), c->head_dim, rows, c->batch);
    // No more blocks than there can be tiles: items are at most one a sequence and head more than whole blocks of rows.
    const uint64_t items = static_cast<uint64_t>(c->kv_heads) * (c->batch + rows / p.shape.rows);
    const uint64_t tiles = static_cast<uint64_t>(capacity_of(c)) / p.shape.tile + 2, most = ar::kTreeMaxBlocks;
    p.blocks = static_cast<int>(items >= most || items * tiles >= most ? most : items * tiles);
    p.slot_rows = static_cast<int>(rows < static_cast<uint64_t>(p.shape.rows) ? rows : p.shape.rows);
    p.slot_floats = (static_cast<size_t>(p.slot_rows) * (c->head_dim + 2) + 3) / 4 * 4;
    p.part_at = (p.blocks * sizeof(ar::TreeJob) + 255) / 256 * 256;
    p.bytes = p.part_at + (2 * p.blocks * p.slot_floats * sizeof(float) + 255) / 256 * 256;
    return p;
}

// ar_kv_append, and with `axes` > 0 ar_kv_append_axes.
int append(const ar_kv_cache* cache, const ar_append_params* p, int axes, size_t axis_stride, const unsigned char* pair_axis,
           ar_stream_t stream)
{
    const ar_kv_cache own = without_idle_strides(cache);
    const ar_kv_cache* const c = &own;
    if (int st = check_sizes(c))
        return st;
    if (p == nullptr)
        return AR_ERR_INVALID_ARG;
    if (int st = check_dtypes(p->dtype, c->dtype))
        return st;
    const bool has_q = p->q != nullptr;
    const size_t d = static_cast<size_t>(c->head_dim);
    if (p->tokens < 0 || (has_q && p->q_heads < 1) || (p->seq_start == nullptr && p->tokens != c->batch) ||
        p->rotary_dim < 0 || p->rotary_dim % 2 != 0 || p->rotary_dim > c->head_dim || !std::isfinite(p->rotary_scale) ||
        (p->rotary_dim > 0 && p->inv_freq == nullptr))
        return AR_ERR_INVALID_ARG;
    if (axes > 0) {
        if (axes > 1 && axis_stride < static_cast<size_t>(p->tokens))
            return AR_ERR_INVALID_ARG;
        for (int j = 0; j < p->rotary_dim / 2; ++j)
            if (pair_axis == nullptr || pair_axis[j] >= axes)
                return AR_ERR_INVALID_ARG;
    }
    if (has_q && p->q_heads > kMaxHeads)
        return AR_ERR_UNSUPPORTED;
    if (p->tokens == 0)
        return AR_OK;
    const size_t e = static_cast<size_t>(esize_of(p->dtype)), ce = static_cast<size_t>(cache_esize_of(c->dtype));
    if (!pointers_ok(c) || !element_ok(p->k, e) || !element_ok(p->v, e) || c->batch < 1 ||
        (has_q && !(element_ok(p->q, e) && element_ok(p->q_out, e))) || !aligned(p->seq_start, 4) ||
        !aligned(p->positions, 4) || !aligned(p->inv_freq, 4) || (axes > 0 && p->positions == nullptr))
        return AR_ERR_INVALID_ARG;
    if (p->tokens > 1 && (p->k_stride < d * c->kv_heads || p->v_stride < d * c->kv_heads ||
                          (has_q && (p->q_stride < d * p->q_heads || p->q_out_stride < d * p->q_heads))))
        return AR_ERR_INVALID_ARG;

    ar::AxesAppendArgs a{};
    a.q = p->q;
    a.k = p->k;
    a.v = p->v;
    a.q_out = p->q_out;
    a.k_pages = c->k;
    a.v_pages = c->v;
    a.table = c->page_table;
    a.lengths = c->lengths;
    a.seq_start = p->seq_start;
    a.positions = p->positions;
    a.inv_freq = p->inv_freq;
    a.q_stride = p->tokens > 1 ? p->q_stride : 0;
    a.k_stride = p->tokens > 1 ? p->k_stride : 0;
    a.v_stride = p->tokens > 1 ? p->v_stride : 0;
    a.q_out_stride = p->tokens > 1 ? p->q_out_stride : 0;
    a.page_stride = c->page_stride;
    a.token_stride = c->token_stride;
    a.head_stride = c->head_stride;
    a.capacity = static_cast<uint64_t>(c->max_pages) * static_cast<uint64_t>(c->page_size);
    a.pages = c->pages;
    a.page_size = c->page_size;
    a.table_stride = c->table_stride;
    a.batch = c->batch;
    a.tokens = p->tokens;
    a.q_heads = has_q ? p->q_heads : 0;
    a.kv_heads = c->kv_heads;
    a.head_dim = c->head_dim;
    a.half = p->rotary_dim / 2;
    a.interleaved = p->interleaved != 0;
    a.rotary_scale = p->rotary_scale;
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;

    // The vector path: every row and head starts on a vector, the rotated part and its halves are whole vectors.
    const size_t lanes = 16 / e;
    const auto whole = [&](size_t stride) { return stride % lanes == 0; };
    const bool vec = whole(d) && whole(a.interleaved ? 2 * a.half : a.half) && aligned(p->k, 16) && aligned(p->v, 16) &&
                     whole(a.k_stride) && whole(a.v_stride) && aligned(c->k, lanes * ce) && aligned(c->v, lanes * ce) &&
                     whole(c->page_stride) && whole(c->token_stride) && whole(c->head_stride) &&
                     (!has_q || (aligned(p->q, 16) && aligned(p->q_out, 16) && whole(a.q_stride) && whole(a.q_out_stride)));
    const int per = vec ? static_cast<int>(lanes) : 1;
    // A unit of a head whose pairs lie apart is a pair of vectors; the rest of it are single ones.
    a.head_units = c->head_dim / per - (a.interleaved && vec ? 0 : a.half / per);
    a.v_units = c->head_dim / per;
    a.head_magic = magic_of(a.head_units);
    a.v_magic = magic_of(a.v_units);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (axes > 0) {
        a.axes = axes;
        a.axis_stride = axes > 1 ? axis_stride : 0;
        for (int j = 0; j < a.half; ++j)
            a.pair_axis[j >> 4] |= static_cast<uint32_t>(pair_axis[j]) << 2 * (j & 15);
        return status_of(by_dtypes(p->dtype, c->dtype, [&](auto t, auto ct) {
            return ar::launch_append<decltype(t), decltype(ct)>(a, vec, s);
        }));
    }
    const ar::AppendArgs& plain = a;
    return status_of(by_dtypes(p->dtype, c->dtype, [&](auto t, auto ct) {
        return ar::launch_append<decltype(t), decltype(ct)>(plain, vec, s);
    }));
}

// More blocks than a launch can have are a call that is not supported, and no failure of CUDA's.
int moved_status(cudaError_t e) { return e == cudaErrorInvalidConfiguration ? AR_ERR_UNSUPPORTED : status_of(e); }

// The largest unit of 16 bytes or less that all of these are whole multiples of.
int unit_of(std::initializer_list<uint64_t> all)
{
    int unit = 16;
    for (const uint64_t x : all)
        while (x % unit != 0)
            unit /= 2;
    return unit;
}

// Lists the layers' buffers, each once, and returns how many they are; 0 where one is missing or misaligned.
int fill_layers(ar::Layers* to, void* const* k, void* const* v, int layers, size_t esize, uint64_t* together)
{
    *together = 0;
    if (k == nullptr || v == nullptr)
        return 0;
    for (int i = 0; i < layers; ++i) {
        if (!element_ok(k[i], esize) || !element_ok(v[i], esize))
            return 0;
        *together |= reinterpret_cast<uintptr_t>(k[i]) | reinterpret_cast<uintptr_t>(v[i]);
    }
    return ar::distinct_buffers(to, k, v, layers);
}

// Whether [a, a + n) and [b, b + m) share an element; either may be NULL.
bool overlap(const int* a, uint64_t n, const int* b, uint64_t m)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a != nullptr && b != nullptr && x < y + 4 * m && y < x + 4 * n;
}

}  // namespace

extern "C" {

int ar_kv_append(const ar_kv_cache* cache, const ar_append_params* p, ar_stream_t stream)
{
    return append(cache, p, 0, 0, nullptr, stream);
}

int ar_kv_append_axes(const ar_kv_cache* cache, const ar_append_params* p, int axes, size_t axis_stride,
                      const unsigned char* pair_axis, ar_stream_t stream)
{
    if (axes < 1 || axes > AR_MAX_AXES)
        return AR_ERR_INVALID_ARG;
    return append(cache, p, axes, axis_stride, pair_axis, stream);
}

int ar_kv_compact(const ar_kv_cache* cache, void* const* k, void* const* v, int layers, const int* kept, size_t kept_stride,
                  int most_kept, const int* seq_start, int drafted, int* new_lengths, ar_stream_t stream)
{
    const ar_kv_cache own = without_idle_strides(cache);
    const ar_kv_cache* const c = &own;
    if (int st = check_layers(c, layers, true))
        return st;
    if (most_kept < 0 || (seq_start == nullptr && drafted < 0) ||
        (c->batch > 1 && kept_stride < static_cast<size_t>(most_kept)))
        return AR_ERR_INVALID_ARG;
    if (c->batch == 0)
        return AR_OK;
    const uint64_t e = static_cast<uint64_t>(cache_esize_of(c->dtype)), batch = static_cast<uint64_t>(c->batch);
    ar::CompactArgs a{};
    uint64_t pointers;
    const int buffers = fill_layers(&a.to, k, v, layers, e, &pointers);
    if (buffers == 0 || !element_ok(c->page_table, 4) || !element_ok(c->lengths, 4) ||
        !aligned(seq_start, 4) || !element_ok(new_lengths, 4) || (most_kept > 0 && !element_ok(kept, 4)))
        return AR_ERR_INVALID_ARG;
    a.kept_stride = c->batch > 1 ? kept_stride : 0;
    if (overlap(new_lengths, batch, c->lengths, batch) || overlap(new_lengths, batch, seq_start, batch + 1) ||
        overlap(new_lengths, batch, kept, (batch - 1) * a.kept_stride + most_kept) ||
        overlap(new_lengths, batch, c->page_table, (batch - 1) * c->table_stride + c->max_pages))
        return AR_ERR_INVALID_ARG;
    a.table = c->page_table;
    a.lengths = c->lengths;
    a.seq_start = seq_start;
    a.kept = kept;
    a.new_lengths = new_lengths;
    a.page_stride = c->page_stride * e;
    a.token_stride = c->token_stride * e;
    a.head_stride = c->head_stride * e;
    a.capacity = static_cast<uint64_t>(c->max_pages) * static_cast<uint64_t>(c->page_size);
    a.drafted = drafted;
    a.most_kept = most_kept;
    a.batch = c->batch;
    a.pages = c->pages;
    a.page_size = c->page_size;
    a.table_stride = c->table_stride;
    const int unit = unit_of({pointers, a.page_stride, a.token_stride, a.head_stride, c->head_dim * e});
    a.inner = static_cast<uint32_t>(c->head_dim * e / unit);
    a.head_units = a.inner * static_cast<uint32_t>(c->kv_heads);
    a.units = a.head_units * static_cast<uint32_t>(buffers);
    return moved_status(ar::launch_compact(a, unit, reinterpret_cast<cudaStream_t>(stream)));
}

int ar_kv_copy_pages(const ar_kv_cache* cache, void* const* k, void* const* v, int layers, const int* src, const int* dst,
                     int pairs, ar_stream_t stream)
{
    const ar_kv_cache own = without_idle_strides(cache);
    const ar_kv_cache* const c = &own;
    if (int st = check_layers(c, layers, false))
        return st;
    if (pairs < 0)
        return AR_ERR_INVALID_ARG;
    if (pairs == 0)
        return AR_OK;
    const uint64_t e = static_cast<uint64_t>(cache_esize_of(c->dtype));
    ar::CopyArgs a{};
    uint64_t pointers;
    const int buffers = fill_layers(&a.to, k, v, layers, e, &pointers);
    if (buffers == 0 || !element_ok(src, 4) || !element_ok(dst, 4))
        return AR_ERR_INVALID_ARG;
    a.src = src;
    a.dst = dst;
    a.pairs = pairs;
    a.pages = c->pages;
    a.page_stride = c->page_stride * e;
    // The page's bytes as runs that lie side by side: heads and tokens in the order of their strides, joined where dense.
    struct Axis {
        uint64_t n, stride;
    } near{static_cast<uint64_t>(c->kv_heads), c->head_stride * e}, far{static_cast<uint64_t>(c->page_size), c->token_stride * e};
    if (near.n == 1 || (far.n > 1 && far.stride < near.stride)) {
        const Axis x = near;
        near = far;
        far = x;
    }
    uint64_t run = c->head_dim * e;
    if (near.n == 1 || near.stride == run) {
        run *= near.n;
        near = far;
        far = {1, 0};
        if (near.n == 1 || near.stride == run) {
            run *= near.n;
            near = {1, 0};
        }
    }
    const int unit = unit_of({pointers, a.page_stride, near.stride, far.stride, run});
    if (run / unit * near.n * far.n > UINT32_MAX)
        return AR_ERR_UNSUPPORTED;
    a.inner = static_cast<uint32_t>(run / unit);
    a.mid = static_cast<uint32_t>(near.n);
    a.mid_stride = near.stride;
    a.outer_stride = far.stride;
    a.units = static_cast<uint32_t>(run / unit * near.n * far.n);
    return moved_status(ar::launch_copy_pages(a, buffers, unit, reinterpret_cast<cudaStream_t>(stream)));
}

size_t ar_paged_attention_workspace_size(const ar_kv_cache* cache, int q_heads)
{
    const ar_kv_cache own = without_idle_strides(cache);
    const ar_kv_cache* const c = &own;
    if (check_attention(c, q_heads) != AR_OK)
        return 0;
    const size_t blocks = static_cast<size_t>(attention_blocks(c, q_heads));
    const size_t slot = static_cast<size_t>(slot_floats_of(c, q_heads)) * sizeof(float);
    return (attention_items(c, q_heads) * sizeof(int2) + 255) / 256 * 256 + (2 * blocks * slot + 255) / 256 * 256;
}

int ar_paged_attention(const ar_kv_cache* cache, const void* q, size_t q_stride, int q_heads, float scale, int window,
                       float softcap, void* out, float* lse, void* workspace, size_t workspace_bytes, int dtype,
                       ar_stream_t stream)
{
    const ar_kv_cache own = without_idle_strides(cache);
    const ar_kv_cache* const c = &own;
    if (int st = check_attention(c, q_heads))
        return st;
    if (int st = check_dtypes(dtype, c->dtype))
        return st;
    if (!std::isfinite(scale) || window < 0 || !std::isfinite(softcap) || softcap < 0.0f)
        return AR_ERR_INVALID_ARG;
    float scale2, softcap2;
    if (!score_factors(scale, c->k_scale, softcap, &scale2, &softcap2))
        return AR_ERR_INVALID_ARG;
    if (c->batch == 0)
        return AR_OK;
    const size_t e = static_cast<size_t>(esize_of(dtype));
    if (!pointers_ok(c) || !element_ok(q, e) || !element_ok(out, e) || !aligned(lse, 4) ||
        (c->batch > 1 && q_stride < static_cast<size_t>(q_heads) * c->head_dim))
        return AR_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(out, 16) ||
        (c->batch > 1 && q_stride * e % 16 != 0) ||
        c->head_dim * e % 16 != 0)
        return AR_ERR_UNSUPPORTED;
    if (workspace == nullptr || !aligned(workspace, 16) ||
        workspace_bytes < ar_paged_attention_workspace_size(c, q_heads))
        return AR_ERR_WORKSPACE;

    const size_t ce = static_cast<size_t>(cache_esize_of(c->dtype));
    ar::AttnArgs a{};
    a.q = static_cast<const char*>(q);
    a.k = static_cast<const char*>(c->k);
    a.v = static_cast<const char*>(c->v);
    a.out = static_cast<char*>(out);
    a.lse = lse;
    a.blocks_of = static_cast<int2*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + (attention_items(c, q_heads) * sizeof(int2) + 255) / 256 * 256);
    a.table = c->page_table;
    a.lengths = c->lengths;
    a.q_stride = c->batch > 1 ? q_stride * e : 0;
    a.page_stride = c->page_stride * ce;
    a.token_stride = c->token_stride * ce;
    a.head_stride = c->head_stride * ce;
    a.table_stride = c->table_stride;
    a.pages = c->pages;
    a.page_size = c->page_size;
    a.batch = c->batch;
    page_division(c->page_size, &a.page_magic, &a.page_shift);
    a.capacity = capacity_of(c);
    a.kv_heads = c->kv_heads;
    a.group = q_heads / c->kv_heads;
    a.group_blocks = group_blocks_of(c, q_heads);
    a.block_heads = ar::attn_block_heads(static_cast<int>(ce));
    a.head_dim = c->head_dim;
    a.window = window;
    a.scale2 = scale2;
    a.softcap = softcap;
    a.softcap2 = softcap2;
    a.v_scale = c->v_scale;
    a.fours_magic = magic_of(c->head_dim / 4);
    a.slot_floats = slot_floats_of(c, q_heads);

    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return AR_ERR_CUDA;
    const int most = attention_blocks(c, q_heads);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return status_of(by_dtypes(dtype, c->dtype, [&](auto t, auto ct) {
        return ar::launch_attention<decltype(t), decltype(ct)>(a, most, sms, s);
    }));
}

size_t ar_tree_attention_workspace_size(const ar_kv_cache* cache, int q_heads, int tokens)
{
    const ar_kv_cache own = without_idle_strides(cache);
    if (check_tree(&own, q_heads, tokens) != AR_OK)
        return 0;
    return tree_plan(&own, q_heads, tokens).bytes;
}

int ar_tree_attention(const ar_kv_cache* cache, const ar_tree_params* p, void* workspace, size_t workspace_bytes, ar_stream_t stream)
{
    const ar_kv_cache own = without_idle_strides(cache);
    const ar_kv_cache* const c = &own;
    if (p == nullptr)
        return AR_ERR_INVALID_ARG;
    if (int st = check_tree(c, p->q_heads, p->tokens))
        return st;
    if (int st = check_dtypes(p->dtype, c->dtype))
        return st;
    float scale2, softcap2;
    if (!std::isfinite(p->scale) || p->window < 0 || !std::isfinite(p->softcap) || p->softcap < 0.0f ||
        !score_factors(p->scale, c->k_scale, p->softcap, &scale2, &softcap2) ||
        (p->mask != nullptr && (p->mask_words < 1 || p->mask_words > 1024)))
        return AR_ERR_INVALID_ARG;
    if (c->batch == 0 ? p->seq_start == nullptr && p->tokens != 0 : p->seq_start == nullptr && p->tokens % c->batch != 0)
        return AR_ERR_INVALID_ARG;
    if (c->batch == 0 || p->tokens == 0)
        return AR_OK;
    const size_t e = static_cast<size_t>(esize_of(p->dtype)), ce = static_cast<size_t>(cache_esize_of(c->dtype));
    if (!pointers_ok(c) || !element_ok(p->q, e) || !element_ok(p->out, e) || !aligned(p->lse, 4) || !aligned(p->seq_start, 4) ||
        !aligned(p->mask, 8) || (p->tokens > 1 && p->q_stride < static_cast<size_t>(p->q_heads) * c->head_dim))
        return AR_ERR_INVALID_ARG;
    if (!aligned(p->q, 16) || !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(p->out, 16) ||
        (p->tokens > 1 && p->q_stride * e % 16 != 0) || c->head_dim * e % 16 != 0)
        return AR_ERR_UNSUPPORTED;
    const TreePlan plan = tree_plan(c, p->q_heads, p->tokens);
    if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < plan.bytes)
        return AR_ERR_WORKSPACE;

    ar::TreeArgs a{};
    a.q = static_cast<const char*>(p->q);
    a.k = static_cast<const char*>(c->k);
    a.v = static_cast<const char*>(c->v);
    a.out = static_cast<char*>(p->out);
    a.lse = p->lse;
    a.jobs = static_cast<ar::TreeJob*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.part_at);
    a.table = c->page_table;
    a.lengths = c->lengths;
    a.seq_start = p->seq_start;
    a.mask = reinterpret_cast<const uint32_t*>(p->mask);
    a.q_stride = p->tokens > 1 ? p->q_stride * e : 0;
    a.page_stride = c->page_stride * ce;
    a.token_stride = c->token_stride * ce;
    a.head_stride = c->head_stride * ce;
    a.table_stride = c->table_stride;
    a.pages = c->pages;
    a.page_size = c->page_size;
    a.batch = c->batch;
    page_division(c->page_size, &a.page_magic, &a.page_shift);
    a.capacity = capacity_of(c);
    a.tokens = p->tokens;
    a.each = p->tokens / c->batch;
    a.mask_words = 2 * p->mask_words;
    a.kv_heads = c->kv_heads;
    a.group = p->q_heads / c->kv_heads;
    a.head_dim = c->head_dim;
    a.window = p->window;
    a.scale2 = scale2;
    a.softcap = p->softcap;
    a.softcap2 = softcap2;
    a.v_scale = c->v_scale;
    a.slot_rows = plan.slot_rows;
    a.slot_floats = plan.slot_floats;
    a.stall = tree_stall();
    ar::TreeMaps maps{};
    a.boxes = tree_maps(c, plan.shape.tile, ar::tree_dim(c->head_dim), &maps, &a.token_first);

    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return AR_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return status_of(by_dtypes(p->dtype, c->dtype, [&](auto t, auto ct) {
        return ar::launch_tree<decltype(t), decltype(ct)>(a, maps, plan.shape, plan.blocks, sms, s);
    }));
}

int ar_attention_join(const void* const* partials, const float* const* lse, int R, int rows, int head_dim, void* out,
                      float* lse_out, int dtype, ar_stream_t stream)
{
    if (R < 1 || R > AR_MAX_RANKS || rows < 0 || head_dim < 1)
        return AR_ERR_INVALID_ARG;
    const int esize = esize_of(dtype);
    if (esize == 0)
        return AR_ERR_UNSUPPORTED;
    if (rows == 0)
        return AR_OK;
    if (partials == nullptr || lse == nullptr || !element_ok(out, esize) || !aligned(lse_out, 4))
        return AR_ERR_INVALID_ARG;
    bool packed = aligned(out, 16);
    ar::JoinArgs a{};
    for (int r = 0; r < R; ++r) {
        if (!element_ok(partials[r], esize) || !element_ok(lse[r], 4) || lse[r] == lse_out)
            return AR_ERR_INVALID_ARG;
        packed = packed && aligned(partials[r], 16);
        a.partials[r] = partials[r];
        a.lse[r] = lse[r];
    }
    a.out = out;
    a.lse_out = lse_out;
    a.R = R;
    a.dim = head_dim;
    a.elements = static_cast<uint64_t>(rows) * static_cast<uint64_t>(head_dim);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return status_of([&] {
        switch (dtype) {
        case AR_FP32: return ar::launch_join<float>(a, packed, s);
        case AR_FP16: return ar::launch_join<__half>(a, packed, s);
        default: return ar::launch_join<__nv_bfloat16>(a, packed, s);
        }
    }());
}

}  // extern "C"
